// Backward pass of the packed forward with grouped heads (attn_bwd_packed):
// dQ, dK, dV by the chain rule of the forward's definition, as in bwd.cu:
//     P = exp(scale Q K^T - LSE), dV = P^T dO, dP = dO V^T, D = rowsum(dO * O),
//     dS = P * (dP - D), dQ = scale dS K, dK = scale dS^T Q,
// with dK and dV of a K/V head summed over the query heads that share it.
//
// Two launches:
//   bwd_prep_kernel   (LSE log2 e, D) of every row, as pairs in the order of
//                     the tiles' rows: [h_kv][token][head of the group].
//   bwd_pack_kernel   one persistent grid of two kinds of CTA, in proportion
//                     to their work, which every CTA works out from the lengths;
//                     some run
//     key tiles       unit = 128 keys of a K/V head, streaming query tiles of
//                     its group (floor(128 / g) tokens times g heads), so the
//                     sum over the group's heads is the product's own sum:
//                     dV += P^T dO and dK += dS^T Q accumulate in TMEM;
//                     the others run
//     query tiles     unit = one query tile, streaming key tiles: dQ += dS K.
// Recomputing S and dP for dQ costs two products more than adding into dQ
// with atomics would, and keeps the result the same from call to call.
//
// Work is dealt out as in the forward (packed_sched.h): a unit cut over
// several CTAs leaves fp32 partial sums, and the range that finishes last adds
// them in the order of the steps.
//
// Rows that are not the sequence's own: P and dS are 0 there by selection (not
// by products, as their inputs may be NaN), the accumulating products stop at
// the 16-row slice that holds the last row, and warp 2 zeroes what is left of
// that slice in the streamed tile.
//
// What bounds it: the chain of a step (S and dP products, P and dS, the sums),
// which the tensor pipe and the elementwise warps share in turns: 1.82 us per
// key-tile step and 1.59 per query-tile step at d = 128 (from s4096 to s8192 by
// the difference, no mask, 2070 MHz), some 3,770 and 3,300 cycles against 2,048
// and 1,536 of products (b1 s8192 h32/8 d128: 2950 us, 932 TFLOP/s on the five
// products of the chain rule; causal 1525 us, 901 TFLOP/s).
//
// Roles (384 threads): warp 0 TMA producer, warp 1 MMA issuer, warp 2 stages
// the steps' (LSE, D) and zeroes tails, warp 3 deals out units, warps 4-11
// elementwise work and epilogue (one TMEM lane per thread, two groups that
// split the columns). TMEM columns as in bwd.cu.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "packed.h"
#include "packed_dev.cuh"
#include "ptx.cuh"

namespace exattn {
namespace {

constexpr int kModeDQ = 0, kModeDKV = 1;
constexpr int kPBwdThreads = 384;
constexpr int kPBwdWarps = 8;  // elementwise warps
constexpr int kStages = 4;     // steps whose (LSE, D) are staged

template <int D>
struct PBwdGeom {
    static constexpr int BT = 128;
    static constexpr int HN = 64;  // a step's scores are handed over in two halves of HN columns
    static constexpr int ROW_BYTES = fwd_row_bytes(D);
    static constexpr int PANELS = (D * 2) / ROW_BYTES;
    static constexpr int PANEL_ELEMS = ROW_BYTES / 2;
    static constexpr int PANEL_BYTES = BT * ROW_BYTES;
    static constexpr int TILE_BYTES = BT * D * 2;
    static constexpr int SLOTS = D == 128 ? 4 : 8;
    static constexpr uint32_t LAYOUT =
        ROW_BYTES == 128 ? kLayoutSw128 : (ROW_BYTES == 64 ? kLayoutSw64 : kLayoutSw32);
    static constexpr uint32_t SBO = 8 * ROW_BYTES;
    static constexpr int TMEM_COLS = 512;
    static constexpr int T_S = 0, T_P = 128, T_A0 = 256, T_A1 = 384;
    static constexpr int T_Q = 384, T_DO = T_Q + D / 2;
    static_assert(T_DO + D / 2 <= TMEM_COLS, "TMEM budget");

    static constexpr int OFF_FIX = 0;
    static constexpr int OFF_RING = 2 * TILE_BYTES;
    static constexpr int OFF_LD = OFF_RING + SLOTS * TILE_BYTES;  // [kStages][2][128] LSE, then D
    static constexpr int OFF_MSG = OFF_LD + kStages * 2 * BT * 4;
    static constexpr int OFF_SUM = OFF_MSG + kMsgSlots * 64;
    static constexpr int OFF_BAR = (OFF_SUM + 2 * 12 * 12 + 15) & ~15;
    static constexpr int BAR_FF = 0, BAR_FE = 1;
    static constexpr int BAR_RF = 2;
    static constexpr int BAR_RE = BAR_RF + SLOTS;
    static constexpr int BAR_SF = BAR_RE + SLOTS;  // [2] a step's S made, its dP made
    static constexpr int BAR_PF = BAR_SF + 2;      // [2] a half's P / dS stored
    static constexpr int BAR_AF = BAR_PF + 2;
    static constexpr int BAR_AE = BAR_AF + 1;
    static constexpr int BAR_LDF = BAR_AE + 1;         // [kStages]
    static constexpr int BAR_LDE = BAR_LDF + kStages;  // [kStages]
    static constexpr int BAR_LAND = BAR_LDE + kStages;  // a tail tile landed
    static constexpr int BAR_ZERO = BAR_LAND + 1;       // its tail zeroed
    static constexpr int BAR_DONE = BAR_ZERO + 1;
    static constexpr int BAR_WG = BAR_DONE + 1;  // the elementwise warps meet (cut units)
    static constexpr int BAR_MF = BAR_WG + 1;
    static constexpr int BAR_ME = BAR_MF + kMsgSlots;
    static constexpr int BAR_MS = BAR_ME + kMsgSlots;  // who shares a cut unit
    static constexpr int NUM_BARS = BAR_MS + kMsgSlots;
    static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;  // TMEM base, abort, joiner
    static constexpr int USED = OFF_MISC + 16;
    static constexpr int MIN_SMEM = 120 * 1024;  // one CTA per SM: it owns all of TMEM
    static constexpr int SMEM_BYTES = (USED > MIN_SMEM ? USED : MIN_SMEM) + 1024;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
};

template <bool BF16>
__device__ __forceinline__ uint32_t pack2q(float lo, float hi) {
    if constexpr (BF16)
        return cvt_pack_bf16(lo, hi);
    else
        return cvt_pack_f16(lo, hi);
}

template <bool BF16>
__device__ __forceinline__ float widen(uint32_t bits) {
    if constexpr (BF16)
        return __uint_as_float(bits << 16);
    else
        return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}

// The last sequence that begins at or before row `tok`, by a warp: 32 starts
// are tried at a time. (Any index where the starts are out of order.)
__device__ __forceinline__ int sequence_of(const SeqArrays &s, int tok) {
    const int lane = threadIdx.x & 31;
    int at = 0, left = s.b;
#pragma unroll 1
    while (left > 1) {
        const int stride = (left + 31) >> 5;
        const bool in = lane * stride < left && (lane == 0 || __ldg(s.cu_q + at + lane * stride) <= tok);
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, in));
        at += k * stride;
        left = min(stride, left - k * stride);
    }
    return at;
}

// (LSE log2 e, D) per row; D / 8 lanes per row, 16 bytes each of O and dO: one
// pass over both, bound by HBM.
//
// D = sum_j P_j dP_j = sum_t dO O. O was rounded to 16 bits, which puts an error
// of up to u |dO| |O| (u = eps / 2) into every dS = P (dP - D) of the row. Where a
// row's weights are spread over many keys |O| is small beside |dP|; where most
// of the weight lies on few keys it is not, and dS itself is small (with all of
// it on one key dS is 0, and the error would be all that is left). Rows that
// see at most kFewKeys keys, which are always of the second kind, form the sum
// over the keys, in fp32. Longer rows that put their weight on one key keep the
// error, as attn_bwd does for every row: telling them apart would take P, which
// only the main kernel has.
constexpr int kFewKeys = 16;

template <int D, bool BF16>
__device__ __forceinline__ float dot8(const uint4 &x, const uint4 &y) {
    const uint32_t ux[4] = {x.x, x.y, x.z, x.w}, uy[4] = {y.x, y.y, y.z, y.w};
    float acc = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        acc = fmaf(widen<BF16>(ux[i] & 0xffffu), widen<BF16>(uy[i] & 0xffffu), acc);
        acc = fmaf(widen<BF16>(ux[i] >> 16), widen<BF16>(uy[i] >> 16), acc);
    }
    return acc;
}

// A block takes `tokens` tokens times `heads` heads (all of them, or a share
// of many), which lie side by side in memory.
template <int D>
struct PrepGeom {
    static constexpr int LPR = D / 8, RPW = 32 / LPR, ROWS = 8 * RPW;
    int heads, tokens, heads_inv;
};
template <int D>
__host__ __device__ __forceinline__ PrepGeom<D> prep_geom(int h) {
    PrepGeom<D> x;
    x.heads = h < PrepGeom<D>::ROWS ? h : PrepGeom<D>::ROWS;
    x.tokens = PrepGeom<D>::ROWS / x.heads;
    x.heads_inv = (65536 + x.heads - 1) / x.heads;  // row / heads = row * heads_inv >> 16, rows <= 128
    return x;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(256) bwd_prep_kernel(const PackBwdArgs a, const PrepGeom<D> geom) {
    griddep_launch_dependents();  // (the main kernel waits before it reads `ld`)
    constexpr int LPR = D / 8;
    const int lane = threadIdx.x & 31, sub = lane % LPR;
    const int row = threadIdx.x / LPR;
    const int t = (row * geom.heads_inv) >> 16;
    const int tok = min(static_cast<int>(blockIdx.x) * geom.tokens + t, a.total_q - 1);
    const int head = min(static_cast<int>(blockIdx.y) * geom.heads + row - t * geom.heads, a.h - 1);
    // (lanes past the end repeat the last row and store nothing)
    const bool live = t < geom.tokens && static_cast<int>(blockIdx.x) * geom.tokens + t < a.total_q &&
                      static_cast<int>(blockIdx.y) * geom.heads + row - t * geom.heads < a.h;
    const int kh = divided(head, a.group_mul, a.group_div), j = head - kh * a.group;
    const int64_t r = static_cast<int64_t>(tok) * a.h + head;
    const uint4 wo = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.o) + r * D + sub * 8);
    const uint4 wd = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.dout) + r * D + sub * 8);
    const float lse2 = a.lse[static_cast<int64_t>(head) * a.total_q + tok] * 1.4426950408889634f;
    // keys this row sees: the warp finds its first row's sequence, lanes of
    // later tokens go on from there
    int seq = sequence_of(a.seqs, __shfl_sync(0xffffffffu, tok, 0));
    while (seq + 1 < a.seqs.b && __ldg(a.seqs.cu_q + seq + 1) <= tok) ++seq;
    const SeqInfo x = seq_info(a.seqs, seq);
    int sees = 0;
    if (tok >= x.q0 && tok < x.q0 + x.sq) sees = a.causal ? min(x.sk, tok - x.q0 + x.sk - x.sq + 1) : x.sk;
    const bool few = sees > 0 && sees <= kFewKeys;
    const int most = __reduce_max_sync(0xffffffffu, few ? sees : 0);

    float acc = dot8<D, BF16>(wo, wd);
#pragma unroll
    for (int off = LPR / 2; off >= 1; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    if (most > 0) {
        const uint16_t *qp = static_cast<const uint16_t *>(a.q) + static_cast<int64_t>(tok) * a.q_stride + head * D;
        const uint16_t *kp = static_cast<const uint16_t *>(a.k) + x.k0 * a.k_stride + kh * D + sub * 8;
        const uint16_t *vp = static_cast<const uint16_t *>(a.v) + x.k0 * a.v_stride + kh * D + sub * 8;
        const uint4 wq = *reinterpret_cast<const uint4 *>(qp + sub * 8);
        float sum = 0.f;
        constexpr int U = 4;  // keys at a time: the loop is bound by the loads' latency
#pragma unroll 1
        for (int i0 = 0; i0 < most; i0 += U) {
            uint4 wk[U], wv[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                wk[u] = wv[u] = make_uint4(0u, 0u, 0u, 0u);
                if (few && i0 + u < sees) {
                    wk[u] = *reinterpret_cast<const uint4 *>(kp + (i0 + u) * a.k_stride);
                    wv[u] = *reinterpret_cast<const uint4 *>(vp + (i0 + u) * a.v_stride);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float s = dot8<D, BF16>(wq, wk[u]), dp = dot8<D, BF16>(wd, wv[u]);
#pragma unroll
                for (int off = LPR / 2; off >= 1; off >>= 1) {
                    s += __shfl_xor_sync(0xffffffffu, s, off);
                    dp += __shfl_xor_sync(0xffffffffu, dp, off);
                }
                if (few && i0 + u < sees) sum = fmaf(fast_exp2(s * a.scale_log2 - lse2), dp, sum);
            }
        }
        if (few) acc = sum;
    }
    if (live && sub == 0)
        a.ld[(static_cast<int64_t>(kh) * a.total_q + tok) * a.group + j] = make_float2(lse2, acc);
}

// Rows of a unit's last streamed tile that are the sequence's own, and
// whether the slice of 16 that holds the last of them needs zeroing.
template <int MODE>
__device__ __forceinline__ int tail_rows(const volatile UnitMsg &x, const PackBwdArgs &a) {
    const int last = x.step0 + x.nstep - 1;
    if constexpr (MODE == kModeDQ) return min(128, x.sk - last * 128);
    return min(a.tile_tokens, x.sq - last * a.tile_tokens) * a.group;
}
template <int MODE>
__device__ __forceinline__ bool tail_zeroed(int rows, const PackBwdArgs &a) {
    // (rows of a query tile past its tokens * group are zero from the start)
    return rows < (MODE == kModeDQ ? 128 : a.tile_tokens * a.group) && (rows & 15) != 0;
}

template <int D, int MODE>
__device__ __forceinline__ void pbwd_producer(const CUtensorMap *tq, const CUtensorMap *tk, const CUtensorMap *tv,
                                              const CUtensorMap *tdo, uint32_t sbase, const UnitMsg *msgs,
                                              const PackBwdArgs &a, const WaitGuard &g) {
    using G = PBwdGeom<D>;
    auto bar = [&](int i) { return sbase + G::OFF_BAR + 8u * i; };
    const uint32_t q_bytes = G::PANELS * a.tile_tokens * a.group * G::ROW_BYTES;
    const uint64_t keep = policy_evict_last();  // streamed tiles are read again by other units
    // one panel of a query tile (rows: token * group + head) or of a key tile
    auto load_q = [&](uint32_t dst, const CUtensorMap *map, uint32_t b, int p, int head, int tok) {
        tma_load_4d_hint(dst + p * G::PANEL_BYTES, map, b, p * G::PANEL_ELEMS, 0, head, tok, keep);
    };
    auto load_k = [&](uint32_t dst, const CUtensorMap *map, uint32_t b, int p, int head, int key) {
        tma_load_4d_hint(dst + p * G::PANEL_BYTES, map, b, p * G::PANEL_ELEMS, head, key, 0, keep);
    };
    int it_u = 0, n_issued = 0;
    bool ok = true;
    UnitMsg x;
    for (; ok && take_unit<false>(&x, it_u, msgs, bar(G::BAR_MF), bar(G::BAR_ME), g, 17); ++it_u) {
        if (!await(bar(G::BAR_FE), (it_u & 1) ^ 1, g, 1)) break;
        mbar_arrive_expect_tx(bar(G::BAR_FF), 2 * (MODE == kModeDQ ? q_bytes : G::TILE_BYTES));
        const uint32_t fix = sbase + G::OFF_FIX;
        for (int p = 0; p < G::PANELS; ++p) {
            if constexpr (MODE == kModeDQ) {
                load_q(fix, tq, bar(G::BAR_FF), p, x.head, x.q0 + x.tok0);
                load_q(fix + G::TILE_BYTES, tdo, bar(G::BAR_FF), p, x.head, x.q0 + x.tok0);
            } else {
                load_k(fix, tk, bar(G::BAR_FF), p, x.head, x.k0 + x.tok0);
                load_k(fix + G::TILE_BYTES, tv, bar(G::BAR_FF), p, x.head, x.k0 + x.tok0);
            }
        }
        for (int i = 0; i < 2 * x.nstep; ++i) {  // step j: K then V, or Q then dO
            const int s = n_issued % G::SLOTS;
            if (!await(bar(G::BAR_RE + s), ((n_issued / G::SLOTS) & 1) ^ 1, g, 2)) {
                ok = false;
                break;
            }
            mbar_arrive_expect_tx(bar(G::BAR_RF + s), MODE == kModeDQ ? G::TILE_BYTES : q_bytes);
            const uint32_t dst = sbase + G::OFF_RING + s * G::TILE_BYTES;
            const int j = x.step0 + (i >> 1);
            for (int p = 0; p < G::PANELS; ++p) {
                if constexpr (MODE == kModeDQ)
                    load_k(dst, (i & 1) ? tv : tk, bar(G::BAR_RF + s), p, x.head, x.k0 + j * G::BT);
                else
                    load_q(dst, (i & 1) ? tdo : tq, bar(G::BAR_RF + s), p, x.head, x.q0 + j * a.tile_tokens);
            }
            ++n_issued;
        }
    }
    // wait (bounded, even after an abort) for the copies still landing
    WaitGuard drain = g;
    uint32_t no_abort = 0;
    drain.abort = &no_abort;
    if (it_u > 0) await(bar(G::BAR_FF), (it_u - 1) & 1, drain, 9);
    for (int n = (n_issued > G::SLOTS ? n_issued - G::SLOTS : 0); n < n_issued; ++n)
        await(bar(G::BAR_RF + n % G::SLOTS), (n / G::SLOTS) & 1, drain, 10);
}

// Warp 2. Key-tile units: each step's (LSE, D) into shared memory, steps
// ahead of their use. Both: a unit's last streamed tile, once it has landed,
// gets zeros in the rows past the sequence that the accumulating products
// still read (K in the query-tile kind, Q and dO in the key-tile kind).
template <int D, int MODE>
__device__ __forceinline__ void pbwd_stage(uint8_t *smem, uint32_t sbase, const UnitMsg *msgs, const PackBwdArgs &a,
                                           const WaitGuard &g) {
    using G = PBwdGeom<D>;
    auto bar = [&](int i) { return sbase + G::OFF_BAR + 8u * i; };
    const int lane = threadIdx.x & 31;
    constexpr int CPR = G::ROW_BYTES / 16;
    int step = 0, zeroed = 0;
    if (MODE == kModeDKV) griddep_wait();  // (LSE, D) are there
    UnitMsg x;
    for (int n = 0; take_unit<true>(&x, n, msgs, bar(G::BAR_MF), bar(G::BAR_ME), g, 17); ++n) {
        if constexpr (MODE == kModeDKV) {
            const float2 *rows = a.ld + (static_cast<int64_t>(x.head) * a.total_q + x.q0) * a.group;
            for (int j = 0; j < x.nstep; ++j) {
                const int s = (step + j) % kStages, tok = (x.step0 + j) * a.tile_tokens;
                const int live = min(a.tile_tokens, x.sq - tok) * a.group;
                float2 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = lane + 32 * i;
                    v[i] = r < live ? __ldcg(rows + static_cast<int64_t>(tok) * a.group + r)
                                    : make_float2(INFINITY, 0.f);
                }
                bool ok = await(bar(G::BAR_LDE + s), (((step + j) / kStages) & 1) ^ 1, g, 20);
                if (!__all_sync(0xffffffffu, ok)) return;
                float *buf = reinterpret_cast<float *>(smem + G::OFF_LD) + s * 2 * G::BT;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    buf[lane + 32 * i] = v[i].x;
                    buf[G::BT + lane + 32 * i] = v[i].y;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(G::BAR_LDF + s));
            }
        }
        if (x.nstep > 0) {
            const int rows = tail_rows<MODE>(x, a);
            if (tail_zeroed<MODE>(rows, a)) {
                const bool ok = await(bar(G::BAR_LAND), zeroed & 1, g, 15);
                ++zeroed;
                if (!__all_sync(0xffffffffu, ok)) return;
                const int per_panel = (((rows + 15) & ~15) - rows) * CPR;
                for (int w = 0; w < (MODE == kModeDQ ? 1 : 2); ++w) {
                    const int item = 2 * (step + x.nstep - 1) + w, slot = item % G::SLOTS;
                    // (the issuer has seen it land and holds the slot)
                    const bool okl = await(bar(G::BAR_RF + slot), (item / G::SLOTS) & 1, g, 16);
                    if (!__all_sync(0xffffffffu, okl)) return;
                    const uint32_t base = sbase + G::OFF_RING + slot * G::TILE_BYTES + rows * G::ROW_BYTES;
                    for (int c = lane; c < per_panel * G::PANELS; c += 32) {
                        const int p = c / per_panel;
                        st_shared_zero16(base + p * G::PANEL_BYTES + (c - p * per_panel) * 16);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(G::BAR_ZERO));
            }
        }
        step += x.nstep;
    }
}

template <int D, int MODE, bool BF16>
__device__ __forceinline__ void pbwd_mma(uint32_t sbase, uint32_t tmem, const UnitMsg *msgs, const PackBwdArgs &a,
                                         const WaitGuard &g) {
    using G = PBwdGeom<D>;
    auto bar = [&](int i) { return sbase + G::OFF_BAR + 8u * i; };
    constexpr uint32_t idesc_s = mma_idesc_f16(G::BT, G::BT, BF16, false, false);
    constexpr uint32_t idesc_acc = mma_idesc_f16(G::BT, D, BF16, false, true);
    const uint64_t fix_k = smem_desc(sbase + G::OFF_FIX, 16, G::SBO, G::LAYOUT);
    const uint64_t ring_k = smem_desc(sbase + G::OFF_RING, 16, G::SBO, G::LAYOUT);
    const uint64_t ring_mn = smem_desc(sbase + G::OFF_RING, G::PANEL_BYTES, G::SBO, G::LAYOUT);
    constexpr uint32_t tile16 = G::TILE_BYTES >> 4;

    // S (w = 0) or dP (w = 1) of a step: a fixed tile (A: from TMEM in the
    // query-tile kind) times a streamed tile (B, K-major), over the head dim
    auto issue_s = [&](auto which, int slot) {
        constexpr int w = decltype(which)::value;
        const uint64_t b = ring_k + slot * tile16;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const int p = (kk * 16) / G::PANEL_ELEMS;
            const int off = ((kk * 16) % G::PANEL_ELEMS) * 2;
            const uint32_t o16 = (p * G::PANEL_BYTES + off) >> 4;
            if constexpr (MODE == kModeDQ)
                mma_ts(tmem + (w ? G::T_P : G::T_S), tmem + (w ? G::T_DO : G::T_Q) + kk * 8, b + o16, idesc_s,
                       kk > 0 ? 1u : 0u);
            else
                mma_ss(tmem + (w ? G::T_P : G::T_S), fix_k + (w ? tile16 : 0u) + o16, b + o16, idesc_s,
                       kk > 0 ? 1u : 0u);
        }
        mma_commit(bar(G::BAR_SF + w));
    };
    using IsS = std::integral_constant<int, 0>;
    using IsP = std::integral_constant<int, 1>;
    // acc (+)= A[TMEM: 128 rows x HN, 16-bit] times rows [h HN, h HN + HN) of
    // a streamed tile (MN-major), up to row `rows`. The group that made
    // columns [32g, 32g + 32) of the half packed them into its columns
    // [32g, 32g + 16). Whole halves are the case that counts: without a
    // condition per product (with one, a product took 150 cycles to issue
    // instead of 64).
    auto acc_half = [&](uint32_t dst, uint32_t a_tmem, uint64_t b_mn, auto half, int rows, bool first) {
        constexpr int h = decltype(half)::value;
        if (rows >= (h + 1) * G::HN) {
#pragma unroll
            for (int kk = 0; kk < G::HN / 16; ++kk)
                mma_ts(dst, a_tmem + h * G::HN + (kk >> 1) * 32 + (kk & 1) * 8,
                       b_mn + (((h * G::HN + kk * 16) * G::ROW_BYTES) >> 4), idesc_acc,
                       (!first || kk > 0) ? 1u : 0u);
        } else {
#pragma unroll 1
            for (int kk = 0; h * G::HN + kk * 16 < rows; ++kk)
                mma_ts(dst, a_tmem + h * G::HN + (kk >> 1) * 32 + (kk & 1) * 8,
                       b_mn + (((h * G::HN + kk * 16) * G::ROW_BYTES) >> 4), idesc_acc,
                       (!first || kk > 0) ? 1u : 0u);
        }
    };
    auto wait_ring = [&](int gs, int &sa, int &sb) {
        const int na = 2 * gs, nb = na + 1;
        sa = na % G::SLOTS;
        sb = nb % G::SLOTS;
        return await(bar(G::BAR_RF + sa), (na / G::SLOTS) & 1, g, 5) &&
               await(bar(G::BAR_RF + sb), (nb / G::SLOTS) & 1, g, 6);
    };

    // (the whole warp follows the control flow; one lane issues)
    int it_u = 0, base = 0, zeroed = 0;
    bool ok = true;
    UnitMsg x;
#pragma unroll 1
    for (; ok && take_unit<true>(&x, it_u, msgs, bar(G::BAR_MF), bar(G::BAR_ME), g, 17); ++it_u) {
        ok = await(bar(G::BAR_FF), it_u & 1, g, 4);
        const int count = x.nstep;
        if (count == 0) {  // nothing to add: the accumulators count as made
            ok = ok && await(bar(G::BAR_AE), (it_u & 1) ^ 1, g, 7);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            if (elect_one()) {
                mma_commit(bar(G::BAR_FE));
                mma_commit(bar(G::BAR_AF));
            }
            continue;
        }
        const int rows_tail = tail_rows<MODE>(x, a);
        const bool zero_tail = tail_zeroed<MODE>(rows_tail, a);
        const int rows_full = MODE == kModeDQ ? G::BT : a.tile_tokens * a.group;
        int sa = 0, sb = 0;
        ok = ok && wait_ring(base, sa, sb);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
        sa = uniform(sa);
        sb = uniform(sb);
        if (elect_one()) {
            if constexpr (MODE == kModeDQ) {
                // Q and dO into TMEM after the last unit's S / dP products (same
                // thread, in order); their shared tiles are then free
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const int p = (kk * 16) / G::PANEL_ELEMS;
                    const int off = ((kk * 16) % G::PANEL_ELEMS) * 2;
                    const uint32_t o16 = (p * G::PANEL_BYTES + off) >> 4;
                    tmem_cp_128x256b(tmem + G::T_Q + kk * 8, fix_k + o16);
                    tmem_cp_128x256b(tmem + G::T_DO + kk * 8, fix_k + tile16 + o16);
                }
                mma_commit(bar(G::BAR_FE));
            }
            issue_s(IsS{}, sa);
            issue_s(IsP{}, sb);
        }
#pragma unroll 1
        for (int j = 0; j < count; ++j) {
            const int gs = base + j;
            int na = sa, nb = sb;  // ring slots of step j + 1
            const bool last = j == count - 1;
            if (last && zero_tail) {
                if (elect_one()) mbar_arrive(bar(G::BAR_LAND));
                ok = await(bar(G::BAR_ZERO), zeroed & 1, g, 11);
                ++zeroed;
            }
            const int rows = uniform(last ? rows_tail : rows_full);
            // first half: added up while the warps work on the second
            ok = ok && await(bar(G::BAR_PF), gs & 1, g, 8);
            // (the unit's first addition overwrites the accumulators: the last
            // unit's epilogue must have read them out)
            if (j == 0) ok = ok && await(bar(G::BAR_AE), (it_u & 1) ^ 1, g, 7);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            tc_fence_after();
            if (elect_one()) {
                if constexpr (MODE == kModeDQ) {
                    acc_half(tmem + G::T_A0, tmem + G::T_S, ring_mn + sa * tile16, IsS{}, rows, j == 0);
                } else {
                    acc_half(tmem + G::T_A0, tmem + G::T_S, ring_mn + sb * tile16, IsS{}, rows, j == 0);
                    acc_half(tmem + G::T_A1, tmem + G::T_P, ring_mn + sa * tile16, IsS{}, rows, j == 0);
                }
            }
            if (!last) ok = wait_ring(gs + 1, na, nb);
            // second half, then the next step's S as soon as what it overwrites
            // has been read, and its dP: the warps begin with S
            ok = ok && await(bar(G::BAR_PF + 1), gs & 1, g, 8);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            tc_fence_after();
            na = uniform(na);
            nb = uniform(nb);
            if (elect_one()) {
                if constexpr (MODE == kModeDQ) {
                    acc_half(tmem + G::T_A0, tmem + G::T_S, ring_mn + sa * tile16, IsP{}, rows, false);
                    if (!last) issue_s(IsS{}, na);
                } else {
                    acc_half(tmem + G::T_A0, tmem + G::T_S, ring_mn + sb * tile16, IsP{}, rows, false);
                    if (!last) issue_s(IsS{}, na);
                    acc_half(tmem + G::T_A1, tmem + G::T_P, ring_mn + sa * tile16, IsP{}, rows, false);
                }
                mma_commit(bar(G::BAR_RE + sa));
                mma_commit(bar(G::BAR_RE + sb));
                if (!last) {
                    issue_s(IsP{}, nb);
                } else {
                    if constexpr (MODE == kModeDKV) mma_commit(bar(G::BAR_FE));
                    mma_commit(bar(G::BAR_AF));
                }
            }
            sa = na;
            sb = nb;
        }
        base += count;
    }
    if (elect_one()) mma_commit(bar(G::BAR_DONE));
    WaitGuard drain = g;
    uint32_t no_abort = 0;
    drain.abort = &no_abort;
    await(bar(G::BAR_DONE), 0, drain, 12);
}

// COLS columns of one fp32 TMEM row, scaled, as 16-bit values at dst, or as
// they are at part (a cut unit's partial sum). Rows lie far apart, so every
// lane's store is a line of its own: 32-byte stores where dst allows them
// (16-byte ones took 3,600 cycles per query tile at d = 128, half of a unit's
// fixed cost).
template <int COLS, bool BF16>
__device__ __forceinline__ void store_acc(uint32_t taddr, float mul, uint16_t *dst, float *part, bool out,
                                          bool zero) {
    constexpr int CH = COLS < 32 ? COLS : 32;
    const bool al32 = (reinterpret_cast<uintptr_t>(dst) & 31u) == 0;
#pragma unroll 1
    for (int c0 = 0; c0 < COLS; c0 += CH) {
        uint32_t v[CH];
        if constexpr (CH == 32)
            tmem_ld32(taddr + c0, *reinterpret_cast<uint32_t(*)[32]>(v));
        else
            tmem_ld16(taddr + c0, *reinterpret_cast<uint32_t(*)[16]>(v));
        tmem_wait_ld();
        if (!out) continue;
        if (part != nullptr) {
#pragma unroll
            for (int i = 0; i < CH / 8; ++i)
                st_global_v8(part + c0 + 8 * i, *reinterpret_cast<const uint32_t(*)[8]>(&v[8 * i]));
            continue;
        }
        uint32_t pk[CH / 2];
#pragma unroll
        for (int i = 0; i < CH / 2; ++i) {
            float lo, hi;
            f2_split(f2_mul(f2_make(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), f2_make(mul, mul)),
                     lo, hi);
            pk[i] = zero ? 0u : pack2q<BF16>(lo, hi);
        }
        if (al32) {
#pragma unroll
            for (int i = 0; i < CH / 16; ++i)
                st_global_v8(dst + c0 + 16 * i, *reinterpret_cast<const uint32_t(*)[8]>(&pk[8 * i]));
        } else {
#pragma unroll
            for (int i = 0; i < CH / 8; ++i)
                reinterpret_cast<uint4 *>(dst + c0)[i] =
                    make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
        }
    }
}

// Adds a cut unit's partial sums of one accumulator in the order of its
// ranges and stores the result: D / 4 lanes per row, 4 rows per thread at a
// time. part(p): range p's rows; dst(row): where a row goes.
template <int D, bool BF16, class Part, class Dst>
__device__ __forceinline__ void join_sums(int nparts, int rows, float mul, Part part, Dst dst) {
    constexpr int LPR = D / 4, RPW = 32 / LPR, R = 4;
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - 4;  // elementwise warp
    const int sub = lane % LPR;
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += kPBwdWarps * RPW * R) {
        int row[R];
        float4 acc[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            row[i] = r0 + (i * kPBwdWarps + w) * RPW + lane / LPR;
            acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll 1
        for (int p = 0; p < nparts; ++p) {
            const float *base = part(p);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (row[i] >= rows) continue;
                const float4 v = __ldcg(reinterpret_cast<const float4 *>(base + static_cast<int64_t>(row[i]) * D) + sub);
                acc[i].x += v.x;
                acc[i].y += v.y;
                acc[i].z += v.z;
                acc[i].w += v.w;
            }
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (row[i] < rows)
                *reinterpret_cast<uint2 *>(dst(row[i]) + 4 * sub) =
                    make_uint2(pack2q<BF16>(acc[i].x * mul, acc[i].y * mul),
                               pack2q<BF16>(acc[i].z * mul, acc[i].w * mul));
    }
}

template <int D, int MODE, bool BF16>
__device__ __forceinline__ void pbwd_compute(uint8_t *smem, uint32_t sbase, uint32_t tmem, const UnitMsg *msgs,
                                             int q4, int cg, int cta, const PackBwdArgs &a, const WaitGuard &g) {
    using G = PBwdGeom<D>;
    auto bar = [&](int i) { return sbase + G::OFF_BAR + 8u * i; };
    const uint32_t lane = threadIdx.x & 31;
    const int row = q4 * 32 + lane;  // TMEM lane = row of the unit's tile
    const uint32_t lanes = static_cast<uint32_t>(q4 * 32) << 16;
    const float c = a.scale_log2;
    const int row_tok = (row * a.group_inv) >> 16, row_head = row - row_tok * a.group;
    volatile int *joiner = reinterpret_cast<volatile int *>(smem + G::OFF_MISC + 8);
    int step = 0, met = 0;
    if (MODE == kModeDQ) griddep_wait();  // (LSE, D) are there
    for (int it_u = 0;; ++it_u) {
        const volatile UnitMsg *x = wait_unit(it_u, msgs, bar(G::BAR_MF), g, 17);
        if (x == nullptr) return;
        const int count = x->nstep;
        // query-tile kind: this row's token, its LSE (log2) and D, and the
        // keys it sees; key-tile kind: this row's key
        const int at = x->tok0 + (MODE == kModeDQ ? row_tok : row);
        const bool out = MODE == kModeDQ ? (row_tok < a.tile_tokens && at < x->sq) : at < x->sk;
        float lse2 = INFINITY, drow = 0.f;
        int sees = 0;  // (DQ) keys seen from the unit's first step on
        int from = 0;  // (DKV) first query token that sees this key, from the unit's first step on
        if constexpr (MODE == kModeDQ) {
            if (out) {
                const float2 v = __ldcg(a.ld + (static_cast<int64_t>(x->head) * a.total_q + x->q0 + at) * a.group +
                                       row_head);
                lse2 = v.x;
                drow = v.y;
                sees = (a.causal ? min(x->sk, at + x->sk - x->sq + 1) : x->sk) - x->step0 * G::BT;
            }
        } else {
            from = a.causal ? at - (x->sk - x->sq) - x->step0 * a.tile_tokens : 0;
        }
        const int own_keys = x->sk - x->step0 * G::BT;  // (DQ) from the unit's first step on
        const int rows_left = MODE == kModeDKV ? x->sq - x->step0 * a.tile_tokens : 0;  // tokens
        for (int j = 0; j < count; ++j, ++step) {
            const float *ldbuf = nullptr;
            int cmin = 0, cmax = G::BT;  // (DKV) the step's columns [cmin, cmax) see this key
            if constexpr (MODE == kModeDKV) {
                const bool okl = await(bar(G::BAR_LDF + step % kStages), (step / kStages) & 1, g, 21);
                if (!__all_sync(0xffffffffu, okl)) return;
                ldbuf = reinterpret_cast<const float *>(smem + G::OFF_LD) + (step % kStages) * 2 * G::BT;
                cmin = min(max(from - j * a.tile_tokens, 0), a.tile_tokens) * a.group;
                cmax = min(rows_left - j * a.tile_tokens, a.tile_tokens) * a.group;
            } else {
                cmax = sees - j * G::BT;
            }
            // 0: every place is the sequence's own and seen; 1: some are hidden by
            // the causal mask; 2: some are not the sequence's own
            int kind = __any_sync(0xffffffffu, cmin > 0 || cmax < G::BT) ? 1 : 0;
            if (MODE == kModeDKV ? cmax < G::BT : own_keys - j * G::BT < G::BT) kind = 2;
            kind = uniform(kind);
            const bool ok = await(bar(G::BAR_SF), step & 1, g, 13);
            if (!__all_sync(0xffffffffu, ok)) return;
            tc_fence_after();
            // a half: P from S, then dS from dP, columns [c0, c0 + 32)
            auto half = [&](auto kind_of, int h) {
                constexpr int KIND = decltype(kind_of)::value;
                const int c0 = h * G::HN + 32 * cg;
                const uint32_t tS = tmem + lanes + G::T_S + c0, tP = tmem + lanes + G::T_P + c0;
                const float4 *ld4 = reinterpret_cast<const float4 *>(ldbuf) + (c0 >> 2);
                uint32_t sv[32], pv[32];
                float *p = reinterpret_cast<float *>(sv);
                // bit i: column c0 + i is seen
                uint32_t seen = ~0u;
                if constexpr (KIND != 0) {
                    const int lo = min(max(cmin - c0, 0), 32), hi = min(max(cmax - c0, 0), 32);
                    seen = static_cast<uint32_t>((1ull << hi) - (1ull << min(lo, hi)));
                }
                tmem_ld32(tS, sv);
                tmem_wait_ld();
                // hidden places get P = 0 by selection; dS = P (dP - D) is then 0
                // too, unless what is there may be NaN (kind 2)
                if constexpr (MODE == kModeDQ) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        p[i] = fast_exp2(p[i] * c - lse2);
                        if (KIND != 0) p[i] = (seen >> i & 1u) ? p[i] : 0.f;
                    }
                } else {
                    uint32_t pp[16];
#pragma unroll
                    for (int q = 0; q < 8; ++q) {  // four columns per shared-memory read
                        const float4 l4 = ld4[q];
                        const float lv[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int i = 4 * q + e;
                            p[i] = fast_exp2(p[i] * c - lv[e]);
                            if (KIND != 0) p[i] = (seen >> i & 1u) ? p[i] : 0.f;
                        }
                        pp[2 * q] = pack2q<BF16>(p[4 * q], p[4 * q + 1]);
                        pp[2 * q + 1] = pack2q<BF16>(p[4 * q + 2], p[4 * q + 3]);
                    }
                    tmem_st16(tS, pp);
                }
                if (h == 0) {
                    const bool okp = await(bar(G::BAR_SF + 1), step & 1, g, 13);
                    if (!__all_sync(0xffffffffu, okp)) return false;
                    tc_fence_after();
                }
                tmem_ld32(tP, pv);
                tmem_wait_ld();
                uint32_t pd[16];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    float dv[4] = {drow, drow, drow, drow}, dr[4];
                    if constexpr (MODE == kModeDKV) {
                        const float4 d4 = ld4[(G::BT >> 2) + q];
                        dv[0] = d4.x;
                        dv[1] = d4.y;
                        dv[2] = d4.z;
                        dv[3] = d4.w;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = 4 * q + e;
                        dr[e] = p[i] * (__uint_as_float(pv[i]) - dv[e]);
                        if (KIND == 2) dr[e] = (seen >> i & 1u) ? dr[e] : 0.f;
                    }
                    pd[2 * q] = pack2q<BF16>(dr[0], dr[1]);
                    pd[2 * q + 1] = pack2q<BF16>(dr[2], dr[3]);
                }
                tmem_st16(MODE == kModeDQ ? tS : tP, pd);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(G::BAR_PF + h));
                    if (MODE == kModeDKV && h == 1) mbar_arrive(bar(G::BAR_LDE + step % kStages));
                }
                return true;
            };
            bool done;
            if (kind == 0) {
                done = half(std::integral_constant<int, 0>{}, 0) && half(std::integral_constant<int, 0>{}, 1);
            } else if (kind == 1) {
                done = true;
#pragma unroll 1
                for (int h = 0; h < 2 && done; ++h) done = half(std::integral_constant<int, 1>{}, h);
            } else {
                done = true;
#pragma unroll 1
                for (int h = 0; h < 2 && done; ++h) done = half(std::integral_constant<int, 2>{}, h);
            }
            if (!done) return;
        }

        // ---------------------------------------------------- epilogue
        const bool ok = await(bar(G::BAR_AF), it_u & 1, g, 14);
        if (!__all_sync(0xffffffffu, ok)) return;
        tc_fence_after();
        // each group stores half of the columns (d = 16: group 0 all of them)
        constexpr int EC = D >= 32 ? D / 2 : D;
        constexpr int ACCS = MODE == kModeDQ ? 1 : 2;
        const int e0 = D >= 32 ? cg * EC : 0;
        const bool mine = D >= 32 || cg == 0;
        const int slot = x->slot;
        float *part = slot < 0 ? nullptr
                               : a.part[MODE] + ((static_cast<int64_t>(2 * cta + slot) * ACCS) * G::BT + row) * D + e0;
        if (mine) {
            if constexpr (MODE == kModeDQ) {
                uint16_t *dst = static_cast<uint16_t *>(a.dq) +
                                (x->q0 + (out ? at : 0)) * a.dq_stride +
                                (x->head * a.group + (out ? row_head : 0)) * D + e0;
                store_acc<EC, BF16>(tmem + lanes + G::T_A0 + e0, a.scale, dst, part, out, count == 0);
            } else {
                const int64_t key = x->k0 + (out ? at : 0);
                store_acc<EC, BF16>(tmem + lanes + G::T_A0 + e0, 1.0f,
                                    static_cast<uint16_t *>(a.dv) + key * a.dv_stride + x->head * D + e0, part, out,
                                    count == 0);
                store_acc<EC, BF16>(tmem + lanes + G::T_A1 + e0, a.scale,
                                    static_cast<uint16_t *>(a.dk) + key * a.dk_stride + x->head * D + e0,
                                    part == nullptr ? nullptr : part + G::BT * D, out, count == 0);
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(G::BAR_AE));
        if (slot >= 0) {
            // a cut unit: count this range's arrival; the last one adds them
            const bool ok = await(bar(G::BAR_MS + it_u % kMsgSlots), (it_u / kMsgSlots) & 1, g, 23);
            if (!__all_sync(0xffffffffu, ok)) return;
            __threadfence();
            if (!meet(bar(G::BAR_WG), met, g)) return;
            if (threadIdx.x == 128) {
                *joiner = arrive_last(a.arrivals + (MODE == kModeDQ ? gridDim.x : 0) + x->first_part, a.call,
                                      x->nparts);
                __threadfence();
            }
            if (!meet(bar(G::BAR_WG), met, g)) return;
            if (*joiner) {
                __threadfence();
                const int first = x->first_part, n = x->nparts, head = x->head, t0 = x->tok0;
                auto part_of = [&](int acc) {
                    return [=, &a](int p) {
                        return a.part[MODE] +
                               (static_cast<int64_t>(2 * (first + p) + (p == 0 ? 1 : 0)) * ACCS + acc) * G::BT * D;
                    };
                };
                if constexpr (MODE == kModeDQ) {
                    const int64_t q0 = x->q0 + t0;
                    join_sums<D, BF16>(n, min(a.tile_tokens, x->sq - t0) * a.group, a.scale, part_of(0),
                                       [&](int r) {
                                           const int tok = (r * a.group_inv) >> 16;
                                           return static_cast<uint16_t *>(a.dq) + (q0 + tok) * a.dq_stride +
                                                  (head * a.group + r - tok * a.group) * D;
                                       });
                } else {
                    const int64_t k0 = x->k0 + t0;
                    const int rows = min(G::BT, x->sk - t0);
                    join_sums<D, BF16>(n, rows, 1.0f, part_of(0), [&](int r) {
                        return static_cast<uint16_t *>(a.dv) + (k0 + r) * a.dv_stride + head * D;
                    });
                    join_sums<D, BF16>(n, rows, a.scale, part_of(1), [&](int r) {
                        return static_cast<uint16_t *>(a.dk) + (k0 + r) * a.dk_stride + head * D;
                    });
                }
            }
        }
        free_unit(it_u, bar(G::BAR_ME));
    }
}

template <int D, int MODE, bool BF16>
__device__ __forceinline__ void pbwd_run(const CUtensorMap *tq, const CUtensorMap *tk, const CUtensorMap *tv,
                                         const CUtensorMap *tdo, uint8_t *smem, uint32_t sbase, uint32_t tmem,
                                         int cta, int ctas, const PackBwdArgs &a, const WaitGuard &g) {
    using G = PBwdGeom<D>;
    auto bar = [&](int i) { return sbase + G::OFF_BAR + 8u * i; };
    const int warp = threadIdx.x >> 5;
    const UnitMsg *msgs = reinterpret_cast<const UnitMsg *>(smem + G::OFF_MSG);
    if (warp == 0) {
        if ((threadIdx.x & 31) == 0 && !(a.flags & kFlagSkipLoads))
            pbwd_producer<D, MODE>(tq, tk, tv, tdo, sbase, msgs, a, g);
    } else if (warp == 1) {
        pbwd_mma<D, MODE, BF16>(sbase, tmem, msgs, a, g);
    } else if (warp == 2) {
        pbwd_stage<D, MODE>(smem, sbase, msgs, a, g);
    } else if (warp == 3) {
        const LineSum *sums = reinterpret_cast<const LineSum *>(smem + G::OFF_SUM) + MODE * (kPBwdThreads / 32);
        post_units<MODE == kModeDKV>(
            a.seqs, a.line[MODE], [&] { return line_total(sums, kPBwdThreads / 32); },
            reinterpret_cast<UnitMsg *>(smem + G::OFF_MSG), bar(G::BAR_MF), bar(G::BAR_ME), bar(G::BAR_MS), g, 18, cta,
            ctas);
    } else {
        pbwd_compute<D, MODE, BF16>(smem, sbase, tmem, msgs, warp & 3, (warp - 4) >> 2, cta, a, g);
    }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kPBwdThreads, 1)
    bwd_pack_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                    const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tdo,
                    const PackBwdArgs a) {
    using G = PBwdGeom<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (sbase - raw);
    auto bar = [&](int i) { return sbase + G::OFF_BAR + 8u * i; };
    const int warp = threadIdx.x >> 5;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + G::OFF_MISC);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + G::OFF_MISC + 4);
    if (threadIdx.x == 0) {
        for (int i = 0; i < G::NUM_BARS; ++i) {
            uint32_t count = 1;
            if ((i >= G::BAR_PF && i < G::BAR_PF + 2) || i == G::BAR_AE || i == G::BAR_WG ||
                (i >= G::BAR_LDE && i < G::BAR_LDE + kStages))
                count = kPBwdWarps;
            if (i >= G::BAR_ME && i < G::BAR_MS) count = 3 + kPBwdWarps;  // producer, issuer, staging, elementwise warps
            mbar_init(bar(i), count);
        }
        *abort_flag = 0u;
        fence_mbar_init();
        tma_prefetch_desc(&tq);
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
        tma_prefetch_desc(&tdo);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), G::TMEM_COLS);
        tmem_relinquish();
    }
    // query tiles of less than 128 rows: the rest of each ring slot is never
    // written by a copy, and read by the key-tile kind's products
    const int used = a.tile_tokens * a.group;
    if (used < G::BT) {
        constexpr int CPR = G::ROW_BYTES / 16;
        const int per = (G::BT - used) * CPR;
#pragma unroll 1
        for (int i = threadIdx.x; i < per * G::PANELS * G::SLOTS; i += kPBwdThreads) {
            const int panel = i / per;
            st_shared_zero16(sbase + G::OFF_RING + panel * G::PANEL_BYTES + used * G::ROW_BYTES + (i - panel * per) * 16);
        }
        fence_proxy_async_smem();
    }
    // both kinds' work, and from it the CTAs that each gets
    LineSum *sums = reinterpret_cast<LineSum *>(smem + G::OFF_SUM);
    line_sum_warps<0>(a.seqs, a.line[kModeDQ], sums);
    line_sum_warps<1>(a.seqs, a.line[kModeDKV], sums + kPBwdThreads / 32);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(*tmem_slot);
    const WaitGuard g{abort_flag, a.status, kKernBwd};
    const int ctas_kv =
        key_ctas(a.line[kModeDQ], line_total(sums, kPBwdThreads / 32), a.line[kModeDKV],
                 line_total(sums + kPBwdThreads / 32, kPBwdThreads / 32), gridDim.x);
    if (static_cast<int>(blockIdx.x) < ctas_kv)
        pbwd_run<D, kModeDKV, BF16>(&tq, &tk, &tv, &tdo, smem, sbase, tmem, blockIdx.x, ctas_kv, a, g);
    else
        pbwd_run<D, kModeDQ, BF16>(&tq, &tk, &tv, &tdo, smem, sbase, tmem, blockIdx.x - ctas_kv,
                                   gridDim.x - ctas_kv, a, g);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, G::TMEM_COLS);
}

template <int D, bool BF16>
cudaError_t launch_bwd_packed_t(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                                const CUtensorMap &tdo, const PackBwdArgs &a, cudaStream_t stream) {
    using G = PBwdGeom<D>;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && !attr_set[dev]) {
        e = cudaFuncSetAttribute(bwd_pack_kernel<D, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 G::SMEM_BYTES);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    const PrepGeom<D> geom = prep_geom<D>(a.h);
    const dim3 grid((a.total_q + geom.tokens - 1) / geom.tokens, (a.h + geom.heads - 1) / geom.heads);
    bwd_prep_kernel<D, BF16><<<grid, 256, 0, stream>>>(a, geom);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    // A short batch's main kernel starts while the first one runs: its set-up
    // and first copies need nothing from it. A long one's CTAs would be placed as
    // SMs come free, neighbours on the work line far apart, so it waits. Waiting
    // against not, causal, us:
    //   2 Mi values of q   h32/8 d128 b2 s256 36.2 30.9, b1 s512 45.3 42.3;
    //                      h16 d64 b8 s256 37.1 31.6, b1 s2048 73.9 73.8
    //   4 Mi               b4 s256 39.1 35.8, b1 s1024 65.8 66.5;
    //                      b16 s256 52.4 55.3, b2 s2048 126.0 138.6
    //   8 Mi               b8 s256 65.1 60.7, b1 s2048 149.6 159.5;
    //                      b32 s256 98.2 114.1, b1 s8192 657 801
    //   32 Mi              b32 s256 194.5 223.5, b1 s8192 1522 1730
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    const bool early = static_cast<int64_t>(a.total_q) * a.h * D <= (2 << 20);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.ctas));
    cfg.blockDim = dim3(kPBwdThreads);
    cfg.dynamicSmemBytes = G::SMEM_BYTES;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, bwd_pack_kernel<D, BF16>, tq, tk, tv, tdo, a);
}

}  // namespace

cudaError_t launch_bwd_packed(int d, bool bf16, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                              const CUtensorMap &tdo, const PackBwdArgs &a, cudaStream_t stream) {
#define EXATTN_PBWD_CASE(DD)                                                       \
    case DD:                                                                       \
        return bf16 ? launch_bwd_packed_t<DD, true>(tq, tk, tv, tdo, a, stream)    \
                    : launch_bwd_packed_t<DD, false>(tq, tk, tv, tdo, a, stream);
    switch (d) {
        EXATTN_PBWD_CASE(16)
        EXATTN_PBWD_CASE(32)
        EXATTN_PBWD_CASE(64)
        EXATTN_PBWD_CASE(128)
        default: return cudaErrorInvalidValue;
    }
#undef EXATTN_PBWD_CASE
}

}  // namespace exattn
