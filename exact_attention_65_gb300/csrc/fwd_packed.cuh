// Forward attention over packed sequences with grouped heads, sm_103a: whole
// prompts packed one behind the other (fwd_packed.cu), and the new tokens of
// each request over a paged cache (chunk_paged.cu).
//
// The mathematics is the forward's (fwd.cu): S = scale Q K^T, an online
// softmax with a running max and sum per row, O = P V, LSE = m + ln l.
//
// Grouped heads: the g = h / h_kv query heads of a K/V head see the same
// keys, so a 128-row query tile holds floor(128 / g) tokens times those g
// heads (row = token * g + head: one TMA box, as they lie side by side in
// memory). Each K/V byte is read once for all heads of the group, a single
// new token fills g rows instead of one, and the causal staircase of a tile
// is g times flatter. Nothing is padded to a head count.
//
// Units and CTAs: a unit is two such tiles (one in the ONE form, which runs
// where no sequence has more rows than a tile) of a sequence and K/V head
// against its keys in steps of 128. Sequence lengths live on the device, so
// every CTA works its part of the call out for itself (packed_sched.h): equal
// shares of the total work, cut inside a unit where that is needed. A cut
// unit's ranges leave normalised fp32 O_i and LSE_i (log2) in the workspace;
// the range that finishes last joins them in the order of the keys, so the
// result does not depend on who that is.
//
// Roles (384 threads, one CTA per SM): warp 0 TMA producer (a whole warp for
// pages, one box per lane; with V by warp 2 in the ONE form), warps 1 and 2
// issue the MMAs of tile 0 and 1 (ONE: warp 1 S, warp 8 P V), warp 3 deals
// out units, warps 4-7 and 8-11 softmax and epilogue of tile 0 and 1. The two
// issuers take turns: with one thread for both tiles the tensor pipe stood
// still while it waited and counted (b1 s8192 h32 d128, no mask: 888 us with one,
// 754 with two when they came in).
//
// Over a cache held in 4 bits (Q4, two tiles; chunk_q4.cu) four more warps, 12-15,
// take the K and V producer's part: they widen rows from the pages into the ring.
// A step takes 2.05 us there (two requests with 512 tokens over 16384 keys: 246 us,
// over 16-bit pages 262).
//
// V rows of a unit's last tile that lie past the sequence belong to the next
// sequence or are stale; P is 0 there, and 0 * NaN is NaN: the issuers zero
// those below the next multiple of 16, where the P V product stops.
//
// What bounds it: long prompts, the tensor pipe beside the softmax warps' use of
// TMEM: a step of two tiles takes 1.50 us (b1 h32/8 d128 without mask, s4096 to
// s8192 to s16384 by differences: 205, 689, 2647 us, 1341 to 1662 TFLOP/s), some
// 3,000 cycles, of which its products need 2,048 (7777 and 8192 tokens causal:
// 743 to 803 us, 1350 to 1460 TFLOP/s, 71 to 77% of the measured peak); single
// tokens, HBM and the change from unit to unit (64 requests of up to 8192 keys,
// h32/8, 16-key pages: 148 to 160 us, 5.8 to 6.3 TB/s, 86 to 93%); batches of
// short sequences, three things about equally: a unit costs 2.2 to 2.7 us besides
// its steps (units of 1 to 8 steps, 8 and 16 to a CTA), the call some 11 us, and
// the shares are uneven where units are short (16 prompts of 64 to 1500 tokens:
// 80 on the fullest CTA against 70 on average; 127 us, 830 TFLOP/s).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "packed.h"
#include "packed_dev.cuh"
#include "ptx.cuh"
#include "q4.cuh"

namespace exattn {
namespace {

// Bit 13 of a kind::f16 instruction descriptor: negate the A operand.
constexpr uint32_t kNegateA = 1u << 13;

template <int D, bool ONE>
struct PackGeom {
    static constexpr int BM = 128;  // rows of a query tile
    static constexpr int BN = 128;  // keys of a step
    static constexpr int QT = ONE ? 1 : 2;
    static constexpr int ROW_BYTES = fwd_row_bytes(D);
    static constexpr int PANELS = (D * 2) / ROW_BYTES;
    static constexpr int PANEL_ELEMS = ROW_BYTES / 2;
    static constexpr int PANEL_BYTES = BM * ROW_BYTES;
    static constexpr int TILE_BYTES = BM * D * 2;
    // K/V tiles in flight. The single-tile form is fed from HBM: its ring is
    // as deep as shared memory allows, or holds 128 KB at small head dims.
    static constexpr int SLOTS = ONE ? (D == 128 ? 6 : (D == 64 ? 10 : 16)) : (D == 128 ? 5 : 8);
    static constexpr int QBUF = D <= 64 ? 2 : 1;
    static constexpr int Q_BUF_BYTES = QT * TILE_BYTES;
    static constexpr uint32_t LAYOUT =
        ROW_BYTES == 128 ? kLayoutSw128 : (ROW_BYTES == 64 ? kLayoutSw64 : kLayoutSw32);
    static constexpr uint32_t SBO = 8 * ROW_BYTES;
    static constexpr int TMEM_COLS = 512;
    static constexpr int TMEM_TILE_STRIDE = 256;
    static constexpr int TMEM_O_OFF = 128;
    static constexpr int OCH = D < 32 ? D : 32;

    static constexpr int OFF_Q = 0;
    static constexpr int OFF_KV = OFF_Q + QBUF * Q_BUF_BYTES;
    static constexpr int OFF_BAR = OFF_KV + SLOTS * TILE_BYTES;
    static constexpr int BAR_QF = 0;              // [QBUF] Q landed
    static constexpr int BAR_QE = BAR_QF + QBUF;  // [QBUF] Q read
    static constexpr int BAR_KVF = BAR_QE + QBUF;
    static constexpr int BAR_KVE = BAR_KVF + SLOTS;
    static constexpr int BAR_SF = BAR_KVE + SLOTS;  // [2] S made (ONE: of even, odd steps)
    static constexpr int BAR_PF = BAR_SF + 2;       // [2] P stored
    static constexpr int BAR_OF = BAR_PF + 2;       // [2] O complete
    static constexpr int BAR_OE = BAR_OF + 2;       // [2] O read out
    static constexpr int BAR_DONE = BAR_OE + 2;
    static constexpr int BAR_TURN = BAR_DONE + 2;  // [2] the tile's issuer may issue
    static constexpr int BAR_PVD = BAR_TURN + 2;  // ONE: [2] P V of an even, an odd step done
    static constexpr int BAR_MF = BAR_PVD + 2;     // [kMsgSlots] unit message posted
    static constexpr int BAR_ME = BAR_MF + kMsgSlots;
    static constexpr int BAR_MS = BAR_ME + kMsgSlots;  // [kMsgSlots] who shares a cut unit
    static constexpr int BAR_WG = BAR_MS + kMsgSlots;  // [2] a tile's softmax warps meet (cut units)
    static constexpr int NUM_BARS = BAR_WG + 2;
    static constexpr int OFF_MSG = (OFF_BAR + NUM_BARS * 8 + 15) & ~15;
    static constexpr int OFF_SUM = OFF_MSG + kMsgSlots * 64;  // a LineSum per warp
    static constexpr int OFF_MISC = OFF_SUM + 16 * 12;        // TMEM base, abort, joiner[2]
    static constexpr int USED = OFF_MISC + 16;
    static constexpr int MIN_SMEM = 120 * 1024;  // one CTA per SM: it owns all of TMEM
    static constexpr int SMEM_BYTES = (USED > MIN_SMEM ? USED : MIN_SMEM) + 1024;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
};

// Threads and registers of a CTA. Over a 4-bit cache four more warps widen its
// rows to 16 bits.
template <bool Q4>
struct PackThreads {
    static constexpr int COUNT = Q4 ? 512 : 384;
    static constexpr int REGS_LAUNCH = Q4 ? 128 : 168;
    static constexpr int REGS_CONTROL = Q4 ? 72 : 96;
    static constexpr int REGS_SOFTMAX = Q4 ? 184 : 200;
    static constexpr int REGS_WIDEN = 72;
    static_assert(4 * REGS_CONTROL + 8 * REGS_SOFTMAX + (Q4 ? 4 * REGS_WIDEN : 0) <= COUNT / 32 * REGS_LAUNCH,
                  "register split");
};

template <bool BF16>
__device__ __forceinline__ uint32_t pack2p(float lo, float hi) {
    if constexpr (BF16)
        return cvt_pack_bf16(lo, hi);
    else
        return cvt_pack_f16(lo, hi);
}

// Query tiles of a unit that hold tokens of the sequence.
template <int QT>
__device__ __forceinline__ int live_tiles(const volatile UnitMsg &x, const PackArgs &a) {
    return x.sq - x.tok0 > a.tile_tokens ? QT : 1;
}

// The ring of K and V tiles as a warp walks it: K_0, V_0, K_1, V_1, ...
template <int SLOTS>
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++slot == SLOTS) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

// The TMA producer: Q and the K and V tiles, through one ring in the order K_0,
// V_0, K_1, V_1, ... A thread issues a box every 100 cycles or so, and a tile
// of 16-key pages is 16 boxes at d = 128, more than a step from HBM takes; so
// the paged one-tile form has two producer warps, one for Q and K and one for
// V (WHICH 0 and 1; 2: both).
template <int D, bool PAGED, bool ONE, int WHICH>
__device__ __forceinline__ void pack_producer(const CUtensorMap *tq, const CUtensorMap *tk,
                                              const CUtensorMap *tv, uint32_t sbase, const UnitMsg *msgs,
                                              const PackArgs &a, const WaitGuard &g) {
    using G = PackGeom<D, ONE>;
    auto bar = [&](int i) { return sbase + G::OFF_BAR + 8u * i; };
    const int lane = threadIdx.x & 31;
    const uint32_t q_box = a.tile_tokens * a.group * G::ROW_BYTES;  // bytes of one panel of a Q tile
    // K/V are read again by the sequence's other units, or once in all
    const uint64_t keep = ONE ? policy_evict_first() : policy_evict_last();
    const int nbox = PAGED ? G::BN / a.box_rows : 1;  // 1 .. 8 boxes, one per lane

    int qb = 0;
    uint32_t q_phase = 1;
    Ring<G::SLOTS> ring;
    ring.phase = 1;
    int q_issued = 0, n_issued = 0;  // items that this warp has issued
    bool ok = true;
    UnitMsg x;
#pragma unroll 1
    for (int n = 0; ok && take_unit<PAGED>(&x, n, msgs, bar(G::BAR_MF), bar(G::BAR_ME), g, 17); ++n) {
        const int end = x.step0 + x.nstep;
        // this lane's page of step j, looked up a step ahead
        auto page_of = [&](int j) {
            int page = a.num_pages;  // past the pool: TMA fills with zeros
            const int key = j * G::BN + lane * a.box_rows;
            if (lane < nbox && j < end && key < x.sk)
                page = min(max(__ldg(a.block_table + static_cast<int64_t>(x.seq) * a.max_pages + key / a.page_size),
                               0),
                           a.num_pages - 1);
            return page;
        };
        int page = PAGED ? page_of(x.step0) : 0;
        if (WHICH != 1) {
            if (!PAGED || lane == 0) {
                ok = await(bar(G::BAR_QE + qb), q_phase, g, 1);
                if (ok) {
                    const int n_qt = live_tiles<G::QT>(x, a);
                    mbar_arrive_expect_tx(bar(G::BAR_QF + qb), n_qt * G::PANELS * q_box);
#pragma unroll 1
                    for (int t = 0; t < n_qt; ++t)
#pragma unroll
                        for (int p = 0; p < G::PANELS; ++p)
                            tma_load_4d(sbase + G::OFF_Q + qb * G::Q_BUF_BYTES + t * G::TILE_BYTES +
                                            p * G::PANEL_BYTES,
                                        tq, bar(G::BAR_QF + qb), p * G::PANEL_ELEMS, 0, x.head,
                                        x.q0 + x.tok0 + t * a.tile_tokens);
                }
            }
            if (PAGED) ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            ++q_issued;
            if (++qb == G::QBUF) {
                qb = 0;
                q_phase ^= 1u;
            }
        }
#pragma unroll 1
        for (int j = x.step0; ok && j < end; ++j) {
            const int page_next = PAGED ? page_of(j + 1) : 0;
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv, ring.next()) {
                if (WHICH != 2 && kv != WHICH) continue;
                const int s = ring.slot;
                if (!PAGED || lane == 0) {
                    ok = await(bar(G::BAR_KVE + s), ring.phase, g, 2);
                    if (ok) mbar_arrive_expect_tx(bar(G::BAR_KVF + s), G::TILE_BYTES);
                }
                if (PAGED) ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                const CUtensorMap *map = kv ? tv : tk;
                const uint32_t dst = sbase + G::OFF_KV + s * G::TILE_BYTES;
                if constexpr (PAGED) {
                    if (lane < nbox) {
                        const int prow = (j * G::BN + lane * a.box_rows) % a.page_size;
#pragma unroll
                        for (int p = 0; p < G::PANELS; ++p)
                            tma_load_4d_hint(dst + lane * a.box_rows * G::ROW_BYTES + p * G::PANEL_BYTES, map,
                                             bar(G::BAR_KVF + s), p * G::PANEL_ELEMS, x.head, prow, page, keep);
                    }
                    __syncwarp();
                } else {
#pragma unroll
                    for (int p = 0; p < G::PANELS; ++p)
                        tma_load_4d_hint(dst + p * G::PANEL_BYTES, map, bar(G::BAR_KVF + s), p * G::PANEL_ELEMS,
                                         x.head, x.k0 + j * G::BN, 0, keep);
                }
                ++n_issued;
            }
            page = page_next;
        }
    }
    // Never leave the CTA with a copy still landing in shared memory: wait for
    // the last items of this warp (an item that was not issued leaves its
    // barrier alone, so its wait would run out: only issued ones are waited for).
    if (!PAGED || lane == 0) {
        WaitGuard drain = g;
        uint32_t no_abort = 0;
        drain.abort = &no_abort;
#pragma unroll 1
        for (int i = (q_issued > G::QBUF ? q_issued - G::QBUF : 0); i < q_issued; ++i)
            await(bar(G::BAR_QF + i % G::QBUF), (i / G::QBUF) & 1, drain, 9);
        constexpr int EACH = WHICH == 2 ? 1 : 2;  // this warp's items are every EACH-th
        static_assert(WHICH == 2 || G::SLOTS % 2 == 0, "a slot belongs to one of the two");
#pragma unroll 1
        for (int i = (n_issued > G::SLOTS / EACH ? n_issued - G::SLOTS / EACH : 0); i < n_issued; ++i) {
            const int item = i * EACH + (WHICH == 1 ? 1 : 0);
            await(bar(G::BAR_KVF + item % G::SLOTS), (item / G::SLOTS) & 1, drain, 10);
        }
    }
}

// The 4-bit form's producers. Q comes by TMA, one lane issuing.
template <int D>
__device__ __forceinline__ void pack_q_producer(const CUtensorMap *tq, uint32_t sbase, const UnitMsg *msgs,
                                                const PackArgs &a, const WaitGuard &g) {
    using G = PackGeom<D, false>;
    auto bar = [&](int i) { return sbase + G::OFF_BAR + 8u * i; };
    const uint32_t q_box = a.tile_tokens * a.group * G::ROW_BYTES;
    int qb = 0, q_issued = 0;
    uint32_t q_phase = 1;
    UnitMsg x;
#pragma unroll 1
    for (int n = 0; take_unit<false>(&x, n, msgs, bar(G::BAR_MF), bar(G::BAR_ME), g, 17); ++n) {
        if (!await(bar(G::BAR_QE + qb), q_phase, g, 1)) break;
        const int n_qt = live_tiles<2>(x, a);
        mbar_arrive_expect_tx(bar(G::BAR_QF + qb), n_qt * G::PANELS * q_box);
#pragma unroll 1
        for (int t = 0; t < n_qt; ++t)
#pragma unroll
            for (int p = 0; p < G::PANELS; ++p)
                tma_load_4d(sbase + G::OFF_Q + qb * G::Q_BUF_BYTES + t * G::TILE_BYTES + p * G::PANEL_BYTES, tq,
                            bar(G::BAR_QF + qb), p * G::PANEL_ELEMS, 0, x.head, x.q0 + x.tok0 + t * a.tile_tokens);
        ++q_issued;
        if (++qb == G::QBUF) {
            qb = 0;
            q_phase ^= 1u;
        }
    }
    // never leave the CTA with a copy still landing (as in pack_producer)
    WaitGuard drain = g;
    uint32_t no_abort = 0;
    drain.abort = &no_abort;
#pragma unroll 1
    for (int i = (q_issued > G::QBUF ? q_issued - G::QBUF : 0); i < q_issued; ++i)
        await(bar(G::BAR_QF + i % G::QBUF), (i / G::QBUF) & 1, drain, 9);
}

// A row of codes and scales of one head, as a thread holds it on its way.
template <int D>
struct Q4Row {
    static constexpr int WORDS = D / 8;  // a word of codes is 8 channels
    uint32_t code[WORDS];
    uint32_t scale[(D + 63) / 64];  // a byte for 16 channels

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) code[i] = 0u;
#pragma unroll
        for (int i = 0; i < (D + 63) / 64; ++i) scale[i] = 0u;
    }
    __device__ __forceinline__ void load(const uint8_t *codes, const uint8_t *scales) {
        if constexpr (D >= 32) {
#pragma unroll
            for (int i = 0; i < WORDS / 4; ++i) {
                const uint4 x = __ldg(reinterpret_cast<const uint4 *>(codes) + i);
                code[4 * i] = x.x, code[4 * i + 1] = x.y, code[4 * i + 2] = x.z, code[4 * i + 3] = x.w;
            }
        } else {
            const uint2 x = __ldg(reinterpret_cast<const uint2 *>(codes));
            code[0] = x.x, code[1] = x.y;
        }
        if constexpr (D == 128) {
            const uint2 x = __ldg(reinterpret_cast<const uint2 *>(scales));
            scale[0] = x.x, scale[1] = x.y;
        } else if constexpr (D == 64) {
            scale[0] = __ldg(reinterpret_cast<const uint32_t *>(scales));
        } else if constexpr (D == 32) {
            scale[0] = __ldg(reinterpret_cast<const uint16_t *>(scales));
        } else {
            scale[0] = __ldg(scales);
        }
    }
};

// Four warps widen K and V: thread r takes key r of each step, from the pages
// through registers (both rows a step ahead) into row r of the ring's tile,
// swizzled as TMA would leave it. Values are exact in either type; K takes Q's
// type, V is fp16. Rows past the sequence's end are zeros. A key with a NaN in V
// gets NaN as its K, which the rows that see it come to feel, and zeros in V, whose
// product with a P of 0 would be NaN in the others.
template <int D, bool BF16>
__device__ __forceinline__ void pack_widen(uint32_t sbase, const UnitMsg *msgs, const PackArgs &a,
                                           const WaitGuard &g) {
    using G = PackGeom<D, false>;
    auto bar = [&](int i) { return sbase + G::OFF_BAR + 8u * i; };
    const int r = threadIdx.x & 127;
    const uint32_t row = r * G::ROW_BYTES;
    constexpr int CPR = G::ROW_BYTES / 16;  // 16-byte chunks of a swizzled row: 8, 4 or 2
    const uint32_t swz = CPR == 8 ? r & 7 : CPR == 4 ? (r >> 1) & 3 : (r >> 2) & 1;
    Ring<G::SLOTS> ring;
    ring.phase = 1;
    bool ok = true;
    UnitMsg x;
#pragma unroll 1
    for (int n = 0; ok && take_unit<true>(&x, n, msgs, bar(G::BAR_MF), bar(G::BAR_ME), g, 17); ++n) {
        const int32_t *table = a.block_table + static_cast<int64_t>(x.seq) * a.max_pages;
        const int end = x.step0 + x.nstep;
        Q4Row<D> buf[2];
        // The page and the row in it (-1: none) of this thread's key in the step
        // that is fetched next, looked up a step before (five prompts of 1900
        // tokens: 192 us, 200 with both loads one behind the other)
        int page = 0, at = -1;
        auto look_up = [&](int j) {
            const int key = j * G::BN + r;
            at = -1;
            if (j < end && key < x.sk) {
                const int p = divided(static_cast<uint32_t>(key) >> 4, a.page_mul, a.page_div);
                at = key - p * a.page_size;
                page = __ldg(table + p);
            }
        };
        auto fetch = [&](int kv) {
            buf[kv].clear();
            if (at >= 0) {
                const uint8_t *block =
                    (kv ? a.v4 : a.k4) +
                    (static_cast<int64_t>(min(max(page, 0), a.num_pages - 1)) * a.line.heads + x.head) * a.block4;
                buf[kv].load(block + static_cast<int64_t>(at) * q4_code_bytes(D),
                             block + static_cast<int64_t>(a.page_size) * q4_code_bytes(D) +
                                 static_cast<int64_t>(at) * q4_scale_bytes(D));
            }
        };
        look_up(x.step0);
        fetch(0);
        fetch(1);
        look_up(x.step0 + 1);
#pragma unroll 1
        for (int j = x.step0; ok && j < end; ++j) {
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                ok = ok && await(bar(G::BAR_KVE + ring.slot), ring.phase, g, 2);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                const uint32_t dst = sbase + G::OFF_KV + ring.slot * G::TILE_BYTES + row;
                uint32_t bad = 0;
#pragma unroll
                for (int i = 0; i < (D + 63) / 64; ++i) bad |= q4_scales_nan(buf[1].scale[i]);
                const uint32_t keep = bad == 0 ? 0xffffffffu : 0u;
#pragma unroll
                for (int i = 0; i < Q4Row<D>::WORDS; ++i) {
                    const uint32_t pair = q4_scales_f16(buf[kv].scale[i / 8] >> (16 * (i / 4 % 2)));
                    uint32_t s2 = __byte_perm(pair, 0, i / 2 % 2 ? 0x3232 : 0x1010);
                    s2 = kv == 0 ? s2 | (~keep & 0x7fff7fffu) : s2 & keep;
                    uint32_t w[4];
                    q4_codes_f16(buf[kv].code[i], w);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        w[e] = h2_mul(w[e], s2);
                        if (BF16 && kv == 0) {
                            const float2 f = h2_float2(w[e]);
                            w[e] = cvt_pack_bf16(f.x, f.y);
                        }
                    }
                    st_shared_v4(dst + i / CPR * G::PANEL_BYTES + ((i % CPR) ^ swz) * 16, w);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if ((threadIdx.x & 31) == 0) mbar_arrive(bar(G::BAR_KVF + ring.slot));
                ring.next();
                fetch(kv);
            }
            look_up(j + 2);
        }
    }
}

// The products of a tile and the zeroing of its V tail, as the issuers use
// them: one lane issues, a whole warp zeroes.
template <int D, bool BF16, bool ONE, bool Q4 = false>
struct TileMma {
    using G = PackGeom<D, ONE>;
    uint32_t sbase, idesc_s;
    uint64_t dq, dk, dv;
    // (values of a 4-bit cache are exact in fp16, and P is rounded less there than in bf16)
    static constexpr uint32_t idesc_o = mma_idesc_f16(G::BM, D, BF16 && !Q4, false, true);
    static constexpr uint32_t tile16 = G::TILE_BYTES >> 4;
    static_assert(G::PANELS <= 2, "panels of a tile");

    __device__ __forceinline__ TileMma(uint32_t base, int t, const PackArgs &a) {
        sbase = base;
        // with a negative scale the S MMAs negate Q, so that the softmax always
        // works with a scale >= 0
        idesc_s = mma_idesc_f16(G::BM, G::BN, BF16, false, false) | (a.scale_log2 < 0.f ? kNegateA : 0u);
        dq = smem_desc(base + G::OFF_Q + t * G::TILE_BYTES, 16, G::SBO, G::LAYOUT);  // K-major
        dk = smem_desc(base + G::OFF_KV, 16, G::SBO, G::LAYOUT);                     // K-major
        dv = smem_desc(base + G::OFF_KV, G::PANEL_BYTES, G::SBO, G::LAYOUT);         // MN-major
    }
    // S = Q K^T of Q buffer qbuf and ring slot `slot`, 16 head-dim elements per
    // instruction; turn: the barrier of the other tile's turn, which passes
    // while the last quarter is still to be queued (0: none)
    __device__ __forceinline__ void s(uint32_t tS, int qbuf, int slot, uint32_t turn) const {
        const uint64_t qdesc = dq + ((qbuf * G::Q_BUF_BYTES) >> 4), kdesc = dk + slot * tile16;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const int p = (kk * 16) / G::PANEL_ELEMS;
            const int off = ((kk * 16) % G::PANEL_ELEMS) * 2;
            const uint32_t o16 = (p * G::PANEL_BYTES + off) >> 4;
            if (!ONE && kk == D / 16 * 3 / 4) mbar_arrive(turn);
            mma_ss(tS, qdesc + o16, kdesc + o16, idesc_s, kk > 0 ? 1u : 0u);
        }
    }
    // O (+)= P V over the first `keys` keys of the tile, 16 per instruction
    // (whole tiles without a condition per product)
    __device__ __forceinline__ void pv(uint32_t tO, uint32_t tP, int slot, int keys, bool first) const {
        const uint64_t vdesc = dv + slot * tile16;
        if (keys == G::BN) {
#pragma unroll
            for (int kk = 0; kk < G::BN / 16; ++kk)
                mma_ts(tO, tP + kk * 8, vdesc + ((kk * 16 * G::ROW_BYTES) >> 4), idesc_o,
                       (!first || kk > 0) ? 1u : 0u);
        } else {
#pragma unroll 1
            for (int kk = 0; kk * 16 < keys; ++kk)
                mma_ts(tO, tP + kk * 8, vdesc + ((kk * 16 * G::ROW_BYTES) >> 4), idesc_o,
                       (!first || kk > 0) ? 1u : 0u);
        }
    }
    // zeros into the rows of a landed V tile from `keys` up to a multiple of 16
    __device__ __forceinline__ void zero_tail(int slot, int keys) const {
        constexpr int CPR = G::ROW_BYTES / 16;
        const int per_panel = (((keys + 15) & ~15) - keys) * CPR;
        const uint32_t base = sbase + G::OFF_KV + slot * G::TILE_BYTES + keys * G::ROW_BYTES;
#pragma unroll 1
        for (int c = threadIdx.x & 31; c < per_panel * G::PANELS; c += 32) {
            const int p = c >= per_panel ? 1 : 0;
            st_shared_zero16(base + p * G::PANEL_BYTES + (c - p * per_panel) * 16);
        }
        fence_proxy_async_smem();
        __syncwarp();
    }
    // No MMA of the calling warp may still be running when TMEM is released.
    __device__ __forceinline__ void finish(int bar, const WaitGuard &g) const {
        const uint32_t b = sbase + G::OFF_BAR + 8u * bar;
        if (elect_one()) mma_commit(b);
        WaitGuard drain = g;
        uint32_t no_abort = 0;
        drain.abort = &no_abort;
        await(b, 0, drain, 12);
    }
};

// The ONE form's two issuers, a warp each: S of step j goes to the S columns
// of tile (j & 1) once the P V product that read them last is done, so S_{j+1}
// is made while the softmax works on S_j. One thread for both kinds took 2,350
// cycles per step for its waiting, counting and issuing. K tiles lie in the
// ring's even slots and V tiles in the odd ones (SLOTS is even), so each slot's
// barriers are seen in order by the warp that waits on them.
template <int D, bool BF16>
__device__ __forceinline__ void issue_one_s(uint32_t sbase, uint32_t tmem, const UnitMsg *msgs, const PackArgs &a,
                                            const WaitGuard &g) {
    using G = PackGeom<D, true>;
    static_assert(G::SLOTS % 2 == 0, "K and V in slots of their own");
    auto bar = [&](int i) { return sbase + G::OFF_BAR + 8u * i; };
    const TileMma<D, BF16, true> mma(sbase, 0, a);
    Ring<G::SLOTS> ring;
    int qbuf = 0;
    uint32_t q_phase = 0, used = 0;  // bit i of used: phase of the uses of S columns i
    bool ok = true;
    UnitMsg x;
#pragma unroll 1
    for (int n = 0; ok && take_unit<true>(&x, n, msgs, bar(G::BAR_MF), bar(G::BAR_ME), g, 17); ++n) {
        ok = await(bar(G::BAR_QF + qbuf), q_phase, g, 4);
#pragma unroll 1
        for (int j = 0; ok && j < x.nstep; ++j) {
            const int c = j & 1;
            ok = await(bar(G::BAR_PVD + c), (used >> c & 1u) ^ 1u, g, 22);
            ok = ok && await(bar(G::BAR_KVF + ring.slot), ring.phase, g, 5);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            used ^= 1u << c;
            tc_fence_after();
            const int ks = uniform(ring.slot), qs = uniform(qbuf);
            if (elect_one()) {
                mma.s(tmem + c * G::TMEM_TILE_STRIDE, qs, ks, 0);
                mma_commit(bar(G::BAR_SF + c));
                mma_commit(bar(G::BAR_KVE + ks));
            }
            ring.next();
            ring.next();
        }
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        if (elect_one()) mma_commit(bar(G::BAR_QE + qbuf));
        if (++qbuf == G::QBUF) {
            qbuf = 0;
            q_phase ^= 1u;
        }
    }
    mma.finish(G::BAR_DONE, g);
}

template <int D, bool BF16>
__device__ __forceinline__ void issue_one_pv(uint32_t sbase, uint32_t tmem, const UnitMsg *msgs, const PackArgs &a,
                                             const WaitGuard &g) {
    using G = PackGeom<D, true>;
    auto bar = [&](int i) { return sbase + G::OFF_BAR + 8u * i; };
    const TileMma<D, BF16, true> mma(sbase, 0, a);
    const uint32_t tO = tmem + G::TMEM_O_OFF;
    Ring<G::SLOTS> ring;
    ring.next();               // V_0
    uint32_t p_phase = 0;      // bit 0 and 1: P of even and odd steps
    uint32_t o_phase = 0;      // O handed back
    bool ok = true;
    UnitMsg x;
#pragma unroll 1
    for (int n = 0; ok && take_unit<true>(&x, n, msgs, bar(G::BAR_MF), bar(G::BAR_ME), g, 17); ++n) {
        const int nkv = x.nstep;
        // O is overwritten: the last unit's must have been read out (also where
        // there is no key to see: O's barrier must not run two phases ahead)
        ok = await(bar(G::BAR_OE), o_phase ^ 1u, g, 7);
        o_phase ^= 1u;
#pragma unroll 1
        for (int j = 0; ok && j < nkv; ++j) {
            const int keys = min(G::BN, x.sk - (x.step0 + j) * G::BN);
            ok = await(bar(G::BAR_KVF + ring.slot), ring.phase, g, 6);
            if (keys & 15) {
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                mma.zero_tail(ring.slot, keys);
            }
            ok = ok && await(bar(G::BAR_PF + (j & 1)), p_phase >> (j & 1) & 1u, g, 8);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            p_phase ^= 1u << (j & 1);
            tc_fence_after();
            const int vs = uniform(ring.slot), ukeys = uniform(keys);
            if (elect_one()) {
                mma.pv(tO, tmem + (j & 1) * G::TMEM_TILE_STRIDE, vs, ukeys, j == 0);
                mma_commit(bar(G::BAR_KVE + vs));
                mma_commit(bar(G::BAR_PVD + (j & 1)));
            }
            ring.next();
            ring.next();
        }
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        if (elect_one()) mma_commit(bar(G::BAR_OF));
    }
    mma.finish(G::BAR_DONE + 1, g);
}

// The MMAs of tile t of two.
template <int D, bool BF16, bool Q4>
__device__ __forceinline__ void pack_issue(uint32_t sbase, uint32_t tmem, const UnitMsg *msgs, int t,
                                           const PackArgs &a, const WaitGuard &g) {
    using G = PackGeom<D, false>;
    auto bar = [&](int i) { return sbase + G::OFF_BAR + 8u * i; };
    const TileMma<D, BF16, false, Q4> mma(sbase, t, a);
    Ring<G::SLOTS> ring;
    int qbuf = 0;
    uint32_t q_phase = 0;         // of the Q buffers
    uint32_t p_phase = 0;         // P stored
    uint32_t o_phase = 0;         // O handed back
    uint32_t turn = t ^ 1u;       // tile 0 goes first
    bool ok = true;
    UnitMsg x;
#pragma unroll 1
    for (int n = 0; ok && take_unit<true>(&x, n, msgs, bar(G::BAR_MF), bar(G::BAR_ME), g, 17); ++n) {
        const int nkv = x.nstep;
        ok = await(bar(G::BAR_QF + qbuf), q_phase, g, 4);
        if (!__all_sync(0xffffffffu, ok)) break;
        const uint32_t qe = bar(G::BAR_QE + qbuf);
        const int qs = uniform(qbuf);
        if (++qbuf == G::QBUF) {
            qbuf = 0;
            q_phase ^= 1u;
        }
        const int last_keys = min(G::BN, x.sk - (x.step0 + nkv - 1) * G::BN);  // of the last step
        // The issuers take turns, P V and the next S of one tile together:
        // otherwise the tiles fall into step, their products side by side
        // and then both in the softmax with the tensor pipe idle (b1 s8192
        // h32 d128: 965 us).
        const bool live = t < live_tiles<2>(x, a);
        const uint32_t tS = tmem + t * G::TMEM_TILE_STRIDE;
#pragma unroll 1
        for (int j = 0; ok && j <= nkv; ++j) {
            const int keys = j == nkv ? last_keys : G::BN;  // of step j - 1
            const Ring<G::SLOTS> vr = ring;
            if (j > 0) ring.next();
            const Ring<G::SLOTS> kr = ring;
            if (j < nkv) ring.next();
            // everything the turn needs: V_{j-1} (its tail zeroed), K_j, P_{j-1}
            if (j > 0) {
                ok = await(bar(G::BAR_KVF + vr.slot), vr.phase, g, 6);
                if (!Q4 && live && (keys & 15)) {  // (rows past the end are widened as zeros)
                    if (!__all_sync(0xffffffffu, ok)) break;
                    mma.zero_tail(vr.slot, keys);
                }
            }
            if (j < nkv) ok = ok && await(bar(G::BAR_KVF + kr.slot), kr.phase, g, 5);
            if (live) {
                // the first P V overwrites O: the last unit's must have been
                // read out (also where there is no key to see: O's barrier
                // must not run two phases ahead)
                if (j == (nkv > 0 ? 1 : 0)) ok = ok && await(bar(G::BAR_OE + t), o_phase ^ 1u, g, 7);
                if (j > 0) {
                    ok = ok && await(bar(G::BAR_PF + t), p_phase, g, 8);
                    p_phase ^= 1u;
                }
            }
            ok = ok && await(bar(G::BAR_TURN + t), turn, g, 22);
            turn ^= 1u;
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const int vs = uniform(vr.slot), ks = uniform(kr.slot), ukeys = uniform(keys);
            if (elect_one()) {
                if (live) {
                    if (j > 0) {  // O += P_{j-1} V_{j-1}
                        mma.pv(tS + G::TMEM_O_OFF, tS, vs, ukeys, j == 1);
                        mma_commit(bar(G::BAR_KVE + vs));
                    }
                    if (j < nkv) {
                        mma.s(tS, qs, ks, bar(G::BAR_TURN + (t ^ 1)));
                        mma_commit(bar(G::BAR_SF + t));
                        mma_commit(bar(G::BAR_KVE + ks));
                        if (j == nkv - 1) mma_commit(qe);
                    } else {
                        mma_commit(bar(G::BAR_OF + t));
                        mbar_arrive(bar(G::BAR_TURN + (t ^ 1)));
                        if (nkv == 0) mma_commit(qe);
                    }
                } else {
                    // not this tile's unit: pass, and release the slots (they
                    // are full, so that a release cannot run ahead)
                    mbar_arrive(bar(G::BAR_TURN + (t ^ 1)));
                    if (j > 0) mbar_arrive(bar(G::BAR_KVE + vr.slot));
                    if (j < nkv) mbar_arrive(bar(G::BAR_KVE + kr.slot));
                    if (j == (nkv > 0 ? nkv - 1 : 0)) mbar_arrive(qe);
                }
            }
        }
        if (!live) continue;
        o_phase ^= 1u;
    }
    mma.finish(G::BAR_DONE + t, g);
}

// Joins a cut unit's partial results of one query tile: with M the largest
// LSE_i, l = sum_i 2^(LSE_i - M), O = sum_i 2^(LSE_i - M) O_i / l, LSE = M +
// log2 l. Run by the tile's 128 threads; a row's columns lie over D / 4 lanes
// (16-byte loads). Bound by the latency of loads from L2, so a warp takes R
// rows times P ranges of them at once. Ranges are taken in order with a
// running maximum.
template <int D, bool BF16, int R, int P>
__device__ __forceinline__ void join_rows(int first_part, int nparts, int t, int tiles, int64_t tok0, int head0,
                                          int rows, const PackArgs &a) {
    constexpr int LPR = D / 4, RPW = 32 / LPR;
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 3;
    const int sub = lane % LPR;
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += 4 * RPW * R) {
        float m[R], l[R];
        float4 acc[R];
        int row[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            row[i] = r0 + (i * 4 + w) * RPW + lane / LPR;
            m[i] = -INFINITY;
            l[i] = 0.f;
            acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll 1
        for (int p0 = 0; p0 < nparts; p0 += P) {
            float lp[P][R];
            float4 op[P][R];
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int part = ((2 * (first_part + p0 + p) + (p0 + p == 0 ? 1 : 0)) * tiles + t) * 128;
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    lp[p][i] = -INFINITY;
                    op[p][i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (p0 + p < nparts && row[i] < rows) {
                        lp[p][i] = __ldcg(a.lse_part + part + row[i]);
                        op[p][i] = __ldcg(reinterpret_cast<const float4 *>(a.o_part) + (part + row[i]) * LPR + sub);
                    }
                }
            }
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float mn = fmaxf(m[i], lp[p][i]);
                    const float f = m[i] == -INFINITY ? 0.f : fast_exp2(m[i] - mn);
                    const float e = lp[p][i] == -INFINITY ? 0.f : fast_exp2(lp[p][i] - mn);
                    m[i] = mn;
                    l[i] = l[i] * f + e;
                    acc[i].x = acc[i].x * f + op[p][i].x * e;
                    acc[i].y = acc[i].y * f + op[p][i].y * e;
                    acc[i].z = acc[i].z * f + op[p][i].z * e;
                    acc[i].w = acc[i].w * f + op[p][i].w * e;
                }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (row[i] >= rows) continue;
            const int rt = (row[i] * a.group_inv) >> 16;
            const int64_t tok = tok0 + rt;
            const int head = head0 + row[i] - rt * a.group;
            const float inv = l[i] == 0.f ? 0.f : 1.0f / l[i];
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.o) + (tok * a.h + head) * D + 4 * sub) =
                make_uint2(pack2p<BF16>(acc[i].x * inv, acc[i].y * inv),
                           pack2p<BF16>(acc[i].z * inv, acc[i].w * inv));
            if (sub == 0)
                a.lse[static_cast<int64_t>(head) * a.total_q + tok] =
                    l[i] == 0.f ? -INFINITY : (m[i] + __log2f(l[i])) * 0.69314718055994530942f;
        }
    }
}

template <int D, bool BF16>
__device__ __forceinline__ void pack_join(int first_part, int nparts, int t, int tiles, int64_t tok0, int head0,
                                          int rows, const PackArgs &a) {
    // few rows: the ranges side by side (b1 sk32768, 20 ranges: one at a time
    // took 20 us); many: the rows
    if (rows <= 16)
        join_rows<D, BF16, 1, 8>(first_part, nparts, t, tiles, tok0, head0, rows, a);
    else
        join_rows<D, BF16, 4, 2>(first_part, nparts, t, tiles, tok0, head0, rows, a);
}

template <int D, bool BF16, bool ONE, bool Q4>
__device__ __forceinline__ void pack_softmax(uint8_t *smem, uint32_t sbase, uint32_t tmem, const UnitMsg *msgs,
                                             int t, int q4, const PackArgs &a, const WaitGuard &g) {
    using G = PackGeom<D, ONE>;
    auto bar = [&](int i) { return sbase + G::OFF_BAR + 8u * i; };
    const uint32_t lane = threadIdx.x & 31;
    const int row = q4 * 32 + lane;
    const int row_tok = (row * a.group_inv) >> 16, row_head = row - row_tok * a.group;
    const bool row_used = row_tok < a.tile_tokens;
    const uint32_t tS0 = tmem + t * G::TMEM_TILE_STRIDE + (static_cast<uint32_t>(q4 * 32) << 16);
    const uint32_t tO = tS0 + G::TMEM_O_OFF;
    const float c = fabsf(a.scale_log2);
    // over a 4-bit cache P is fp16 whatever the type, and 2^6 times as large (at
    // most 2^14): its least values are 2^-30 of the reference max
    constexpr bool P_BF16 = BF16 && !Q4;
    constexpr float P_SHIFT = Q4 ? 6.0f : 0.0f;
    int s_cnt = 0, s2_cnt = 0, o_cnt = 0;
    int met = 0;      // meetings of the tile's warps
    volatile int *joiner = reinterpret_cast<volatile int *>(smem + G::OFF_MISC + 8);

    for (int n = 0;; ++n) {
        const volatile UnitMsg *x = wait_unit(n, msgs, bar(G::BAR_MF), g, 17);
        if (x == nullptr) return;
        if (t >= live_tiles<G::QT>(*x, a)) {
            free_unit(n, bar(G::BAR_ME));
            continue;
        }
        const int tok = x->tok0 + t * a.tile_tokens + row_tok;  // this row's token in the sequence
        const bool row_out = row_used && tok < x->sq;
        // A warp without a row of the sequence skips the math but keeps the
        // barrier protocol.
        const bool warp_live = __any_sync(0xffffffffu, row_out);
        // keys of the range this row sees (0 or less: none)
        const int sees = (a.causal ? min(x->sk, tok + x->sk - x->sq + 1) : x->sk) - x->step0 * G::BN;
        const int nstep = x->nstep;

        float m_ref = -INFINITY;  // reference max, log2 units
        float l = 0.f;            // running sum of 2^(s*c - m_ref)
        bool alive = true;
        for (int j = 0; j < nstep; ++j) {
            const bool alt = ONE && (j & 1);  // ONE: odd steps use the second tile's S columns
            const uint32_t tS = alt ? tS0 + G::TMEM_TILE_STRIDE : tS0;
            const bool ok = await(bar(alt ? G::BAR_SF + 1 : G::BAR_SF + t), (alt ? s2_cnt : s_cnt) & 1, g, 13);
            if (alt)
                ++s2_cnt;
            else
                ++s_cnt;
            if (!__all_sync(0xffffffffu, ok)) {
                alive = false;
                break;
            }
            tc_fence_after();
            if (warp_live) {
                const int valid = sees - j * G::BN;
                const int vmax = __reduce_max_sync(0xffffffffu, valid);
                const bool ragged = __any_sync(0xffffffffu, valid < G::BN);
                // the row's max over the tile; `step(mraw)` moves the reference max
                // when a tile exceeds it by more than 8 (log2): P stays at most
                // 2^8, exact in 16 bits as below 1. A row that has seen no key
                // yet keeps m = -inf and alpha 1.
                bool need = false;
                float alpha = 1.0f;
                auto step = [&](float mraw) {
                    // (a scale of 0 makes every score 0: 0 * -inf must not be NaN)
                    const float m_tile = mraw == -INFINITY ? -INFINITY : mraw * c;
                    need = m_tile > m_ref + 8.0f;
                    const float m_new = need ? m_tile : m_ref;
                    if (m_new != -INFINITY) alpha = fast_exp2(m_ref - m_new);
                    m_ref = m_new;
                };
                uint64_t acc2[2] = {0ull, 0ull};
                // P = 2^(s*c - m_ref), rounded to 16 bits for the P V product
                // (the row sum takes the unrounded values), packed in pairs
                // into the S columns
                if (!ragged) {
                    uint32_t sr[G::BN];
                    const float *s = reinterpret_cast<const float *>(sr);
                    float mx[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) mx[i] = -INFINITY;
                    // the max of the first 64 scores runs while the rest load
                    tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
                    tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
                    tmem_wait_ld();
                    tmem_ld32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(&sr[64]));
                    tmem_ld32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(&sr[96]));
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        if (part == 1) tmem_wait_ld();
#pragma unroll
                        for (int i = part * G::BN / 4; i < (part + 1) * G::BN / 4; ++i)
                            mx[i & 3] = max3f(mx[i & 3], s[2 * i], s[2 * i + 1]);
                    }
                    step(fmaxf(max3f(mx[0], mx[1], mx[2]), mx[3]));
                    const float neg_m = Q4 ? P_SHIFT - m_ref : -m_ref;
                    const uint64_t c2 = f2_make(c, c), nm2 = f2_make(neg_m, neg_m);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t pk[G::BN / 4];
#pragma unroll
                        for (int i = 0; i < G::BN / 4; ++i) {
                            const int k0 = half * (G::BN / 2) + 2 * i;
                            float x0, x1;
                            f2_split(f2_fma(f2_make(s[k0], s[k0 + 1]), c2, nm2), x0, x1);
                            const float p0 = fast_exp2(x0);
                            const float p1 = fast_exp2(x1);
                            acc2[i & 1] = f2_add(acc2[i & 1], f2_make(p0, p1));
                            pk[i] = pack2p<P_BF16>(p0, p1);
                        }
                        tmem_st32(tS + half * (G::BN / 4), pk);
                    }
                } else {
                    // A masked or ragged tile, 32 keys at a time: chunks that no
                    // row of the warp sees are skipped, keys the row does not see
                    // get exactly 0. Scores are read twice rather than kept, and
                    // the chunks stay a loop: code four times smaller. (A chunk's
                    // P goes to columns whose scores have been read.)
                    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
                    for (int c0 = 0; c0 < vmax && c0 < G::BN; c0 += 32) {
                        uint32_t sr[32];
                        tmem_ld32(tS + c0, sr);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (c0 + i < valid) mx[i & 1] = fmaxf(mx[i & 1], __uint_as_float(sr[i]));
                    }
                    step(fmaxf(mx[0], mx[1]));
                    const float neg_m = Q4 ? P_SHIFT - m_ref : -m_ref;
                    const uint64_t c2 = f2_make(c, c), nm2 = f2_make(neg_m, neg_m);
#pragma unroll 1
                    for (int c0 = 0; c0 < G::BN; c0 += 32) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) pk[i] = 0u;
                        if (c0 < vmax) {
                            uint32_t sr[32];
                            tmem_ld32(tS + c0, sr);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                float x0, x1;
                                f2_split(f2_fma(f2_make(__uint_as_float(sr[2 * i]), __uint_as_float(sr[2 * i + 1])),
                                                c2, nm2),
                                         x0, x1);
                                const float p0 = fast_exp2(c0 + 2 * i < valid ? x0 : -INFINITY);
                                const float p1 = fast_exp2(c0 + 2 * i + 1 < valid ? x1 : -INFINITY);
                                acc2[i & 1] = f2_add(acc2[i & 1], f2_make(p0, p1));
                                pk[i] = pack2p<P_BF16>(p0, p1);
                            }
                        }
                        tmem_st16(tS + c0 / 2, pk);
                    }
                }
                const bool rescale = j > 0 && __any_sync(0xffffffffu, need);
                if (rescale) {
                    // O row *= alpha once P_{j-1} V_{j-1} is done: S_j's
                    // commit covers it where S_j was issued after it; ONE
                    // issues S_j earlier and waits for that product's own barrier
                    if (ONE) {
                        const bool okv =
                            await(bar(G::BAR_PVD + (alt ? 0 : 1)), ((alt ? s_cnt : s2_cnt) - 1) & 1, g, 15);
                        if (!__all_sync(0xffffffffu, okv)) {
                            alive = false;
                            break;
                        }
                        tc_fence_after();
                    }
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 16) {
                        uint32_t ov[16];
                        tmem_ld16(tO + c0, ov);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                        tmem_st16(tO + c0, ov);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(alt ? G::BAR_PF + 1 : G::BAR_PF + t));
                float a0, a1, a2, a3;
                f2_split(acc2[0], a0, a1);
                f2_split(acc2[1], a2, a3);
                l = l * alpha + ((a0 + a1) + (a2 + a3));
            } else {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(alt ? G::BAR_PF + 1 : G::BAR_PF + t));
            }
        }
        if (!alive) return;

        // ---------------------------------------------------- epilogue
        // A row that saw no key of the range: O = 0, LSE = -inf. (Not told by
        // l > 0: a NaN among the row's inputs has to come out as NaN.)
        const bool empty_row = nstep == 0 || sees <= 0;
        const float inv_l = empty_row ? 0.0f : (Q4 ? a.v_scale4 : 1.0f) / l;
        const int slot = x->slot;
        const bool part = slot >= 0;
        const int64_t grow = x->q0 + (row_out ? tok : 0);
        const int head = x->head * a.group + row_head;
        uint16_t *dst = static_cast<uint16_t *>(a.o) + (grow * a.h + (row_out ? head : 0)) * D;
        const int64_t prow =
            (static_cast<int64_t>(2 * static_cast<int>(blockIdx.x) + max(slot, 0)) * G::QT + t) * 128 + row;
        const bool o_al32 = (reinterpret_cast<uintptr_t>(a.o) & 31u) == 0;
        const bool ok = await(bar(G::BAR_OF + t), o_cnt & 1, g, 14);
        ++o_cnt;
        if (!__all_sync(0xffffffffu, ok)) return;
        tc_fence_after();
        if (warp_live) {
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += G::OCH) {
                uint32_t ov[G::OCH];
                if constexpr (G::OCH == 32)
                    tmem_ld32(tO + c0, *reinterpret_cast<uint32_t(*)[32]>(ov));
                else
                    tmem_ld16(tO + c0, *reinterpret_cast<uint32_t(*)[16]>(ov));
                tmem_wait_ld();
                if (!row_out) continue;
                if (part) {
#pragma unroll
                    for (int i = 0; i < G::OCH; ++i)
                        ov[i] = empty_row ? 0u : __float_as_uint(__uint_as_float(ov[i]) * inv_l);
#pragma unroll
                    for (int i = 0; i < G::OCH / 8; ++i)
                        st_global_v8(a.o_part + prow * D + c0 + 8 * i,
                                     *reinterpret_cast<const uint32_t(*)[8]>(&ov[8 * i]));
                } else {
                    uint32_t pk[G::OCH / 2];
#pragma unroll
                    for (int i = 0; i < G::OCH / 2; ++i) {
                        float lo, hi;
                        f2_split(f2_mul(f2_make(__uint_as_float(ov[2 * i]), __uint_as_float(ov[2 * i + 1])),
                                        f2_make(inv_l, inv_l)),
                                 lo, hi);
                        pk[i] = empty_row ? 0u : pack2p<BF16>(lo, hi);
                    }
                    if (o_al32) {
#pragma unroll
                        for (int i = 0; i < G::OCH / 16; ++i)
                            st_global_v8(dst + c0 + 16 * i, *reinterpret_cast<const uint32_t(*)[8]>(&pk[8 * i]));
                    } else {
#pragma unroll
                        for (int i = 0; i < G::OCH / 8; ++i)
                            reinterpret_cast<uint4 *>(dst + c0)[i] =
                                make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
                    }
                }
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(G::BAR_OE + t));
        const float lse2 = empty_row ? -INFINITY : m_ref + __log2f(l) - P_SHIFT;
        if (!part) {
            if (row_out) a.lse[static_cast<int64_t>(head) * a.total_q + grow] = lse2 * 0.69314718055994530942f;
            free_unit(n, bar(G::BAR_ME));
            continue;
        }
        // A cut unit: count this range's arrival; the last one joins them all.
        {
            const bool ok = await(bar(G::BAR_MS + n % kMsgSlots), (n / kMsgSlots) & 1, g, 23);
            if (!__all_sync(0xffffffffu, ok)) return;
        }
        if (row_out) a.lse_part[prow] = lse2;
        __threadfence();
        if (!meet(bar(G::BAR_WG + t), met, g)) return;
        if (row == 0) {
            joiner[t] = arrive_last(a.arrivals + x->first_part * G::QT + t, a.call, x->nparts);
            __threadfence();
        }
        if (!meet(bar(G::BAR_WG + t), met, g)) return;
        if (joiner[t]) {
            __threadfence();
            const int tile_tok = x->tok0 + t * a.tile_tokens;
            const int toks = min(a.tile_tokens, x->sq - tile_tok);
            pack_join<D, BF16>(x->first_part, x->nparts, t, G::QT, static_cast<int64_t>(x->q0) + tile_tok,
                               x->head * a.group, toks * a.group, a);
        }
        free_unit(n, bar(G::BAR_ME));
    }
}

template <int D, bool BF16, bool PAGED, bool ONE, bool Q4>
__global__ void __launch_bounds__(PackThreads<Q4>::COUNT, 1)
    pack_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                const __grid_constant__ CUtensorMap tv, const PackArgs a) {
    using G = PackGeom<D, ONE>;
    using T = PackThreads<Q4>;
    static_assert(!Q4 || (PAGED && !ONE), "the 4-bit cache has the two-tile form");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (sbase - raw);
    auto bar = [&](int i) { return sbase + G::OFF_BAR + 8u * i; };

    const int warp = threadIdx.x >> 5;
    const uint32_t lane = threadIdx.x & 31;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + G::OFF_MISC);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + G::OFF_MISC + 4);
    UnitMsg *msgs = reinterpret_cast<UnitMsg *>(smem + G::OFF_MSG);
    LineSum *sums = reinterpret_cast<LineSum *>(smem + G::OFF_SUM);

    if (threadIdx.x == 0) {
        for (int i = 0; i < G::NUM_BARS; ++i) {
            uint32_t count = 1;
            if ((i >= G::BAR_PF && i < G::BAR_PF + 2) || (i >= G::BAR_OE && i < G::BAR_OE + 2))
                count = 4;  // the tile's softmax warps
            if (i >= G::BAR_WG) count = 4;
            if (i >= G::BAR_ME && i < G::BAR_MS) count = ONE ? 7 + (PAGED ? 1 : 0) : Q4 ? 15 : 11;  // producers, issuers, softmax warps
            // released by each tile's issuer
            if ((i >= G::BAR_QE && i < G::BAR_KVF) || (i >= G::BAR_KVE && i < G::BAR_SF)) count = G::QT;
            if (Q4 && i >= G::BAR_KVF && i < G::BAR_KVE) count = 4;  // the widening warps
            mbar_init(bar(i), count);
        }
        *abort_flag = 0u;
        fence_mbar_init();
        tma_prefetch_desc(&tq);
        if (!Q4) {
            tma_prefetch_desc(&tk);
            tma_prefetch_desc(&tv);
        }
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), G::TMEM_COLS);
        tmem_relinquish();
    }
    if (a.seqs.b > 32) line_sum_warps<0, Q4>(a.seqs, a.line, sums, a.filter);  // (fewer: post_units does it alone)
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitGuard g{abort_flag, a.status, kKernFwd};

    if (warp < 4) {
        reg_dealloc<T::REGS_CONTROL>();
        if (Q4 && warp == 0) {
            if (lane == 0 && !(a.flags & kFlagSkipLoads)) pack_q_producer<D>(&tq, sbase, msgs, a, g);
        } else if (warp == 0) {
            if ((PAGED || lane == 0) && !(a.flags & kFlagSkipLoads))
                pack_producer<D, PAGED, ONE, PAGED && ONE ? 0 : 2>(&tq, &tk, &tv, sbase, msgs, a, g);
        } else if (warp < 3) {
            if constexpr (!ONE) {
                pack_issue<D, BF16, Q4>(sbase, tmem, msgs, warp - 1, a, g);
            } else {
                if (warp == 1)
                    issue_one_s<D, BF16>(sbase, tmem, msgs, a, g);
                else if constexpr (PAGED)
                    if (!(a.flags & kFlagSkipLoads))
                        pack_producer<D, PAGED, ONE, 1>(&tq, &tk, &tv, sbase, msgs, a, g);
            }
        } else {
            post_units<0, Q4>(
                a.seqs, a.line, [&] { return line_total(sums, T::COUNT / 32); }, msgs, bar(G::BAR_MF),
                bar(G::BAR_ME), bar(G::BAR_MS), g, 18, blockIdx.x, gridDim.x, a.filter);
        }
    } else if (Q4 && warp >= 12) {
        reg_dealloc<T::REGS_WIDEN>();
        if constexpr (Q4)
            if (!(a.flags & kFlagSkipLoads)) pack_widen<D, BF16>(sbase, msgs, a, g);
    } else {
        reg_alloc<T::REGS_SOFTMAX>();
        if (ONE && warp == 8)
            issue_one_pv<D, BF16>(sbase, tmem, msgs, a, g);
        if (warp < 4 + 4 * G::QT)
            pack_softmax<D, BF16, ONE, Q4>(smem, sbase, tmem, msgs, (warp - 4) >> 2, warp & 3, a, g);
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, G::TMEM_COLS);
    // (the few-row kernel before it: what comes behind in the stream waits for this one)
    if (Q4 && threadIdx.x == 0) griddep_wait();
}

template <int D, bool BF16, bool PAGED, bool ONE>
cudaError_t launch_pack_t(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const PackArgs &a,
                          cudaStream_t stream) {
    using G = PackGeom<D, ONE>;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && !attr_set[dev]) {
        e = cudaFuncSetAttribute(pack_kernel<D, BF16, PAGED, ONE, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 G::SMEM_BYTES);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    pack_kernel<D, BF16, PAGED, ONE, false>
        <<<a.ctas, PackThreads<false>::COUNT, G::SMEM_BYTES, stream>>>(tq, tk, tv, a);
    return cudaGetLastError();
}

template <int D, bool PAGED>
cudaError_t launch_pack_d(bool bf16, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                          const PackArgs &a, cudaStream_t stream) {
    if (a.one_tile)
        return bf16 ? launch_pack_t<D, true, PAGED, true>(tq, tk, tv, a, stream)
                    : launch_pack_t<D, false, PAGED, true>(tq, tk, tv, a, stream);
    return bf16 ? launch_pack_t<D, true, PAGED, false>(tq, tk, tv, a, stream)
                : launch_pack_t<D, false, PAGED, false>(tq, tk, tv, a, stream);
}

template <bool PAGED>
cudaError_t launch_pack(int d, bool bf16, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                        const PackArgs &a, cudaStream_t stream) {
    switch (d) {
        case 16: return launch_pack_d<16, PAGED>(bf16, tq, tk, tv, a, stream);
        case 32: return launch_pack_d<32, PAGED>(bf16, tq, tk, tv, a, stream);
        case 64: return launch_pack_d<64, PAGED>(bf16, tq, tk, tv, a, stream);
        case 128: return launch_pack_d<128, PAGED>(bf16, tq, tk, tv, a, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace
}  // namespace exattn
