// Declarations of the packed and paged operators' translation units.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "exattn.h"
#include "internal.h"
#include "packed_sched.h"

namespace exattn {

// ------------------------------------------------------------ packed batches
// The sequences of a packed batch, on the device.
struct SeqArrays {
    const int32_t *cu_q;     // [b + 1] first query row of each sequence
    const int32_t *cu_k;     // [b + 1] first key row (packed K/V); nullptr for a paged cache
    const int32_t *seqlens;  // [b] keys of each sequence (paged cache); nullptr for packed K/V
    int b, total_q;
    int max_k;  // key rows (packed), or the most keys a row of the block table holds (paged)
};
// A sequence with fewer or more query rows than this is another kernel's: no work
// here.
struct SeqFilter {
    int least = 0, most = 0x7fffffff;
};

// Grouped-head forward over packed or paged K/V (fwd_packed.cuh).
struct PackArgs {
    SeqArrays seqs;
    LineShape line;
    void *o;
    float *lse;  // [h, total_q]
    int h, group;     // query heads, query heads per K/V head
    int group_inv;    // row / group = row * group_inv >> 16 for rows below 128
    int tile_tokens;  // tokens of a 128-row query tile: floor(128 / group)
    int total_q;
    int causal;
    int one_tile;  // units of one query tile instead of two
    float scale_log2;
    uint32_t *status;
    uint32_t flags;
    int ctas;
    // cut units: normalised O_i [ctas, 2, tiles, 128, d] and log2 LSE_i
    // [ctas, 2, tiles, 128] (fp32), and an arrival counter per CTA and tile,
    // valid for call number `call` (24 bits)
    float *o_part, *lse_part;
    uint32_t *arrivals;
    uint32_t call;
    // paged K/V
    const int32_t *block_table;
    int page_size, max_pages, num_pages, box_rows;
    // a 4-bit cache (q4.cuh): its pools, bytes of a page of a head, V's scale
    const uint8_t *k4, *v4;
    int64_t block4;
    float v_scale4;
    // ... and tile / (tiles of 16 keys in a page) = tile * page_mul >> page_div
    uint32_t page_mul;
    int page_div;
    // few rows over it (decode_q4.cu): q itself, bytes of a page of all heads
    const void *q;
    int64_t q_stride;
    uint32_t page_bytes;
    SeqFilter filter;  // (over a 4-bit cache)
};
// Query tokens of a 128-row tile, and where work is cut.
inline int pack_tile_tokens(int group) { return 128 / group; }
// ceil(2^16 / group): exact for rows below 128, as 128 * group_inv errs by
// less than 128 / 2^16 < 1 / group.
inline int pack_group_inv(int group) { return (65536 + group - 1) / group; }
// The most the work line of a call can hold, from what the host knows.
struct LineBound {
    int b, total_q;
    int64_t total_k, max_k;  // keys of all sequences, and of one, at most
};
LineShape pack_line(int heads, int group, bool one_tile, bool causal, const LineBound &bound);
LineShape bwd_key_line(int heads, int group, bool causal, const LineBound &bound);
cudaError_t launch_fwd_packed(int d, bool bf16, const CUtensorMap &tq, const CUtensorMap &tk,
                              const CUtensorMap &tv, const PackArgs &a, cudaStream_t stream);
cudaError_t launch_chunk_paged(int d, bool bf16, const CUtensorMap &tq, const CUtensorMap &tk,
                               const CUtensorMap &tv, const PackArgs &a, cudaStream_t stream);
// early: may start while launch_decode_q4()'s kernel before it still runs
cudaError_t launch_chunk_q4(int d, bool bf16, const CUtensorMap &tq, const PackArgs &a, bool early,
                            cudaStream_t stream);
// The most rows (tokens times a group's heads) of a unit of launch_decode_q4()
// with so many rows to a request: 8 or 16, 0 where it has more. Its work is dealt
// to the warps of two CTAs an SM; each leaves up to two ranges' O_i and LSE_i
// [warps, 2, rows], with three counters.
constexpr int decode_q4_rows(int64_t rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 0; }
constexpr int decode_q4_warps(int rows) { return rows == 8 ? 8 : 6; }
constexpr int decode_q4_ctas(int rows) { return 2; }
LineShape decode_q4_line(int heads, int tokens, bool causal, const LineBound &bound);
cudaError_t launch_decode_q4(int d, bool bf16, int rows, const PackArgs &a, cudaStream_t stream);

// Backward of the packed forward (bwd_packed.cu). Index 0: query-tile units
// (dQ), 1: key-tile units (dK, dV).
struct PackBwdArgs {
    SeqArrays seqs;
    LineShape line[2];
    const void *q, *k, *v;  // rows q_stride, k_stride, v_stride elements apart
    int64_t q_stride, k_stride, v_stride;
    const void *o, *dout;  // [total_q, h, d]
    const float *lse;      // [h, total_q]
    float2 *ld;            // workspace [h_kv, total_q, group]: (LSE log2 e, D)
    void *dq, *dk, *dv;
    int64_t dq_stride, dk_stride, dv_stride;  // elements from one token's row to the next
    int h, group, group_inv, tile_tokens, total_q, causal;
    uint32_t group_mul;  // head / group = head * group_mul >> group_div
    int group_div;
    float scale, scale_log2;
    uint32_t *status;
    uint32_t flags;
    int ctas;
    // cut units of each kind: fp32 sums [ctas, 2, accumulators, 128, d], and a
    // counter per CTA (key tiles first), valid for call number `call`
    float *part[2];
    uint32_t *arrivals;
    uint32_t call;
};
LineShape bwd_query_line(int heads, int group, bool causal, const LineBound &bound);
cudaError_t launch_bwd_packed(int d, bool bf16, const CUtensorMap &tq, const CUtensorMap &tk,
                              const CUtensorMap &tv, const CUtensorMap &tdo, const PackBwdArgs &a,
                              cudaStream_t stream);

// ------------------------------------------------------------ paged cache upkeep
struct PlanArgs {
    const int32_t *seqlens, *new_lens;  // [b]
    int32_t *block_table;               // [b, max_pages]
    const int32_t *free_pages;          // [num_free], a stack
    const int32_t *free_count;          // [1]
    int32_t *cu_seqlens_q;              // [b + 1]
    int32_t *seqlens_out;               // [b]
    int64_t *slot_map;                  // [max_tokens]
    int32_t *free_left;                 // [1]
    int b, max_pages, page_size, num_free;
    int64_t max_tokens;
};
cudaError_t launch_paged_plan(const PlanArgs &a, int num_sms, cudaStream_t stream);

struct WriteArgs {
    const uint4 *k, *v;          // rows of `words` 16-byte words, k_stride / v_stride words apart
    const int64_t *slot_map;     // [tokens]
    uint4 *k_pages, *v_pages;    // [slots, words]
    int64_t tokens, k_stride, v_stride, slots;
    int words, step_words;  // words of a row; of the step from one of a thread's words to the next,
    int64_t step_tokens;    //   with its tokens (set by the launch)
};
cudaError_t launch_paged_write(const WriteArgs &a, cudaStream_t stream);

// Rotation and rows into pages (append_paged.cu). Rows and their strides in
// 16-byte words.
struct AppendArgs {
    const uint4 *q, *k, *v;
    uint4 *q_out;
    const float *cos_sin;                // [max_positions, rot]: cosines, then sines
    const int64_t *positions, *slot_map;  // [tokens]
    void *k_pages, *v_pages;
    int64_t tokens, max_positions, slots, q_stride, k_stride, v_stride, q_out_stride;
    int h, h_kv, rot, interleaved, page_size;
    // 4-bit pages: the tensors' scales, six times each, bytes of a page of a head
    // and of its codes
    float k_scale, v_scale, k_six, v_six;
    int64_t block, codes;
    int per_token, per_token_log2;  // set by the launch
};
cudaError_t launch_append(const AppendArgs &a, int d, bool bf16, bool q4, cudaStream_t stream);

// Rows out of a 4-bit cache (append_paged.cu).
struct ReadQ4Args {
    const uint8_t *k_pages, *v_pages;
    const int64_t *slot_map;  // [tokens]
    uint4 *k, *v;             // rows k_stride, v_stride 16-byte words apart
    int64_t tokens, slots, k_stride, v_stride, block, codes;
    int h_kv, page_size;
    int gpr_log2, wide;  // set by the launch
    float k_scale, v_scale;
};
cudaError_t launch_read_q4(const ReadQ4Args &a, int d, bool bf16, cudaStream_t stream);

// 16-bit tensor with four dimensions, innermost first; strides in bytes of
// dimensions 1 to 3.
bool encode_dims(CUtensorMap *map, const void *base, bool bf16, const uint64_t (&dims)[4],
                 const uint64_t (&strides)[3], const uint32_t (&box)[4], CUtensorMapSwizzle swizzle);
CUtensorMapSwizzle fwd_swizzle(int d);
// The current device: its status word and SM count (made ready on first use).
attn_status_t device_info(int *dev, uint32_t **status, int *num_sms);
// Frees what the packed entry points keep per stream on device `dev`.
void packed_release(int dev);

}  // namespace exattn
