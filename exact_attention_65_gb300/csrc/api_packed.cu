// C-ABI layer of the packed and paged operators with grouped heads: argument
// checks, tensor maps, and the workspace of cut units. Declared in
// include/exattn.h.
#include <cmath>
#include <cstdint>
#include <mutex>
#include <vector>

#include "exattn.h"
#include "packed.h"

using namespace exattn;

namespace exattn {

namespace {

// Costs count 2^k steps each where the line would not fit 31 bits.
void fit_line(LineShape *s, const LineBound &x) {
    // units, and steps of a unit, at most
    const double units = (static_cast<double>(s->by_key ? x.total_k : x.total_q) / s->unit_len + x.b) * s->heads;
    const double steps = static_cast<double>(s->by_key ? x.total_q : x.max_k) * s->weight / (1 << s->shift);
    fast_division(s->unit_len, &s->unit_mul, &s->unit_div);
    fast_division(s->step_len, &s->step_mul, &s->step_div);
    for (double w = units * (steps + s->unit_cost + 1); w > 1.0e9; w /= 2) {
        ++s->shift;
        s->unit_cost = s->unit_cost > 1 ? s->unit_cost / 2 : 1;
        s->min_part = s->min_part > 1 ? s->min_part / 2 : 1;
    }
}

}  // namespace

// Where the forward's work is cut (packed_sched.h). A unit's fixed cost (Q,
// first S, epilogue) counts as two steps of 128 keys (one: b2 s8192 h32/8 d128
// causal 783 us, two: 740; measured, it is one and a half). Joining a cut unit
// costs as much as several steps of two tiles, so these are cut only where a
// CTA's share is 16 steps, six away from a unit's ends (16 prompts of 64 to
// 1500 tokens: 145 us with 4 and 2, 132 with 16 and 6); units of one tile, where
// a long cache has to be spread over many CTAs and few rows are joined, from 4
// steps on, two from the ends. These numbers come from calls with work for every
// CTA; a small one is spread too thinly by them (one token over 900 keys on 8
// K/V heads: 64 steps on 16 CTAs, the longest chain 6).
LineShape pack_line(int heads, int group, bool one_tile, bool causal, const LineBound &bound) {
    LineShape s;
    s.heads = heads;
    s.unit_len = pack_tile_tokens(group) * (one_tile ? 1 : 2);
    s.step_len = 128;
    s.causal = causal ? 1 : 0;
    s.by_key = 0;
    s.weight = 1;
    s.shift = 7;
    s.unit_cost = kUnitSteps;
    s.min_steps = one_tile ? 2 : 6;
    s.min_part = one_tile ? 4 : 16;
    fit_line(&s, bound);
    return s;
}

// The backward's query-tile units: one tile against steps of 128 keys.
LineShape bwd_query_line(int heads, int group, bool causal, const LineBound &bound) {
    return pack_line(heads, group, true, causal, bound);
}

// Its key-tile units: 128 keys against tiles of query tokens, whose heads
// make rows of them.
LineShape bwd_key_line(int heads, int group, bool causal, const LineBound &bound) {
    LineShape s;
    s.heads = heads;
    s.unit_len = 128;
    s.step_len = pack_tile_tokens(group);
    s.causal = causal ? 1 : 0;
    s.by_key = 1;
    s.weight = group;
    s.shift = 7;
    s.unit_cost = kUnitSteps;
    s.min_steps = 2;
    s.min_part = 8;
    fit_line(&s, bound);
    return s;
}

}  // namespace exattn

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kDevices = 64;
constexpr int kMaxRows = 0x7fffff00;  // the ends of tiles stay below 2^31
constexpr int64_t kMaxUnits = 1 << 29;  // of a call (fit_line() leaves a unit a cost of 1 at least)

bool misaligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// What the cut units of a call leave for one another, kept per stream: calls
// on a stream are ordered, so each call reuses it. The lock is held until the
// call is enqueued, so that another host thread cannot replace the buffers in
// between. A handle may come back for another stream once its stream is
// destroyed, even with work of that one still to do, so an entry also holds
// the stream's id, which is unique.
struct PackWs {
    cudaStream_t stream;
    unsigned long long id;
    uint32_t *arrivals = nullptr;
    int n_arrivals = 0;
    char *part = nullptr;
    size_t part_bytes = 0;
    uint32_t call = 0;
};
std::vector<PackWs> g_ws[kDevices];
std::mutex g_ws_mu;

struct Workspace {
    std::unique_lock<std::mutex> lock;
    uint32_t *arrivals = nullptr;
    uint32_t call = 0;
    char *part = nullptr;
    void *owned = nullptr;  // a workspace of this call's own, to be freed stream-ordered
};

// n arrival counters and part_bytes of partial results of one call's own, from
// the memory pool.
attn_status_t own_workspace(cudaStream_t stream, size_t count_bytes, size_t part_bytes, Workspace *w) {
    void *p = nullptr;
    if (cudaMallocAsync(&p, count_bytes + part_bytes, stream) != cudaSuccess) {
        cudaGetLastError();
        return ATTN_ERR_NO_MEMORY;
    }
    if (cudaMemsetAsync(p, 0, count_bytes, stream) != cudaSuccess) {
        cudaFreeAsync(p, stream);
        return ATTN_ERR_CUDA;
    }
    w->owned = p;
    w->arrivals = static_cast<uint32_t *>(p);
    w->part = static_cast<char *>(p) + count_bytes;
    w->call = 1;
    return ATTN_OK;
}

// The stream's workspace, grown where it is too small. Streams that cannot have
// one of their own get it for the call alone: one that is being captured (its
// replays are not ordered with the stream's other calls), the per-thread
// default stream (one handle, many streams), and one whose handle was another
// stream's before (what that one still has to do is not ordered with it; its
// entry stays until packed_release()).
attn_status_t get_workspace(int dev, cudaStream_t stream, int n, size_t part_bytes, Workspace *w) {
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(stream, &cs) != cudaSuccess) {
        cudaGetLastError();
        return ATTN_ERR_CUDA;
    }
    const size_t count_bytes = (static_cast<size_t>(n) * sizeof(uint32_t) + 255) / 256 * 256;
    if (cs != cudaStreamCaptureStatusNone || stream == cudaStreamPerThread)
        return own_workspace(stream, count_bytes, part_bytes, w);
    unsigned long long id = 0;
    if (cudaStreamGetId(stream, &id) != cudaSuccess) {
        cudaGetLastError();
        return ATTN_ERR_CUDA;
    }
    w->lock = std::unique_lock<std::mutex>(g_ws_mu);
    PackWs *e = nullptr;
    for (auto &x : g_ws[dev])
        if (x.stream == stream) e = &x;
    if (e == nullptr) {
        PackWs x;
        x.stream = stream;
        x.id = id;
        try {
            g_ws[dev].push_back(x);
        } catch (...) {  // no exception leaves the library
            return ATTN_ERR_NO_MEMORY;
        }
        e = &g_ws[dev].back();
    }
    if (e->id != id) {
        w->lock.unlock();
        return own_workspace(stream, count_bytes, part_bytes, w);
    }
    if (e->n_arrivals < n) {
        void *p = nullptr;
        if (cudaMallocAsync(&p, count_bytes, stream) != cudaSuccess) {
            cudaGetLastError();
            return ATTN_ERR_NO_MEMORY;
        }
        if (cudaMemsetAsync(p, 0, count_bytes, stream) != cudaSuccess) {
            cudaFreeAsync(p, stream);
            return ATTN_ERR_CUDA;
        }
        if (e->arrivals) cudaFreeAsync(e->arrivals, stream);
        e->arrivals = static_cast<uint32_t *>(p);
        e->n_arrivals = n;
    }
    if (e->part_bytes < part_bytes) {
        void *p = nullptr;
        if (cudaMallocAsync(&p, part_bytes, stream) != cudaSuccess) {
            cudaGetLastError();
            return ATTN_ERR_NO_MEMORY;
        }
        if (e->part) cudaFreeAsync(e->part, stream);
        e->part = static_cast<char *>(p);
        e->part_bytes = part_bytes;
    }
    e->call = e->call >= 0xffffffu ? 1 : e->call + 1;
    w->arrivals = e->arrivals;
    w->part = e->part;
    w->call = e->call;
    return ATTN_OK;
}

// Units are counted in 31 bits: those of h_kv heads, of `rows` rows in b
// sequences, unit_len rows at least in each.
attn_status_t check_units(int b, int rows, int unit_len, int h_kv) {
    const int64_t units = rows / unit_len + (b < rows ? b : rows);
    return units * h_kv <= kMaxUnits ? ATTN_OK : ATTN_ERR_UNSUPPORTED;
}

// What every packed attention call checks. Strides are in elements, of the
// token dimension of q, k and v.
attn_status_t check_packed(int b, int total_q, int h, int h_kv, int d, float scale, int dtype) {
    if (b < 1 || total_q < 1 || h < 1 || h_kv < 1) return ATTN_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
    if (dtype != ATTN_FP16 && dtype != ATTN_BF16) return ATTN_ERR_INVALID_ARG;
    if (h % h_kv != 0) return ATTN_ERR_INVALID_ARG;
    if (d != 16 && d != 32 && d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
    if (b > 65535 || h > 65535 || h / h_kv > 128) return ATTN_ERR_UNSUPPORTED;
    if (total_q > kMaxRows) return ATTN_ERR_UNSUPPORTED;
    return check_units(b, total_q, pack_tile_tokens(h / h_kv), h_kv);
}

attn_status_t check_stride(int64_t stride, int64_t row) {
    if (stride < row || stride % 8 != 0) return ATTN_ERR_INVALID_ARG;
    if (stride * 2 >= (1ll << 40)) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

// Rows [total, h, d] with a token stride, read in boxes of `tokens` tokens of
// one K/V head's group of query heads: dims (d, group, h_kv, total).
bool encode_rows(CUtensorMap *map, const void *base, bool bf16, int d, int h, int h_kv, int64_t total,
                 int64_t stride, int tokens) {
    const uint64_t g = h / h_kv, row = static_cast<uint64_t>(d) * 2;
    const uint64_t dims[4] = {static_cast<uint64_t>(d), g, static_cast<uint64_t>(h_kv), static_cast<uint64_t>(total)};
    const uint64_t strides[3] = {row, row * g, static_cast<uint64_t>(stride) * 2};
    const uint32_t box[4] = {static_cast<uint32_t>(fwd_row_bytes(d) / 2), static_cast<uint32_t>(g), 1u,
                             static_cast<uint32_t>(tokens)};
    return encode_dims(map, base, bf16, dims, strides, box, fwd_swizzle(d));
}

// Rows [total, h_kv, d] with a token stride, read 128 at a time: dims (d,
// h_kv, total, 1).
bool encode_keys(CUtensorMap *map, const void *base, bool bf16, int d, int h_kv, int64_t total, int64_t stride) {
    const uint64_t row = static_cast<uint64_t>(d) * 2, st = static_cast<uint64_t>(stride) * 2;
    const uint64_t dims[4] = {static_cast<uint64_t>(d), static_cast<uint64_t>(h_kv), static_cast<uint64_t>(total), 1};
    const uint64_t strides[3] = {row, st, st};
    const uint32_t box[4] = {static_cast<uint32_t>(fwd_row_bytes(d) / 2), 1u, 128u, 1u};
    return encode_dims(map, base, bf16, dims, strides, box, fwd_swizzle(d));
}

// Common part of the two forwards: everything but K and V.
void fill_pack(PackArgs *a, void *o, float *lse, int b, int total_q, int max_seqlen_q, int h, int h_kv,
               int64_t max_k, float scale, bool causal, uint32_t *status, int num_sms) {
    a->o = o;
    a->lse = lse;
    a->h = h;
    a->group = h / h_kv;
    a->tile_tokens = pack_tile_tokens(a->group);
    a->total_q = total_q;
    a->causal = causal ? 1 : 0;
    a->scale_log2 = scale * kLog2e;
    a->status = status;
    a->flags = debug_flags();
    a->ctas = num_sms;
    // Units of one query tile where no sequence is known to hold more.
    const int longest = max_seqlen_q > 0 && max_seqlen_q < total_q ? max_seqlen_q : total_q;
    a->one_tile = longest <= a->tile_tokens ? 1 : 0;
    a->group_inv = pack_group_inv(a->group);
    a->line = pack_line(h_kv, a->group, a->one_tile != 0, causal, LineBound{b, total_q, max_k, max_k});
    a->seqs.b = b;
    a->seqs.total_q = total_q;
    a->block_table = nullptr;
    a->page_size = a->max_pages = a->num_pages = a->box_rows = 0;
}

template <class Launch>
attn_status_t run_pack(PackArgs *a, int dev, int d, cudaStream_t stream, Launch launch) {
    const size_t rows = static_cast<size_t>(a->ctas) * 2 * (a->one_tile ? 1 : 2) * 128;
    Workspace w;
    const attn_status_t st =
        get_workspace(dev, stream, 2 * a->ctas, rows * (static_cast<size_t>(d) + 1) * sizeof(float), &w);
    if (st != ATTN_OK) return st;
    a->arrivals = w.arrivals;
    a->call = w.call;
    a->o_part = reinterpret_cast<float *>(w.part);
    a->lse_part = a->o_part + rows * d;
    const cudaError_t e = launch();
    const cudaError_t ef = w.owned ? cudaFreeAsync(w.owned, stream) : cudaSuccess;
    return (e == cudaSuccess && ef == cudaSuccess) ? ATTN_OK : ATTN_ERR_CUDA;
}

bool overlap(const void *p, size_t np, const void *q, size_t nq) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + nq && b < a + np;
}

}  // namespace

void exattn::packed_release(int dev) {
    if (dev < 0 || dev >= kDevices) return;
    std::lock_guard<std::mutex> lock(g_ws_mu);
    for (auto &x : g_ws[dev]) {
        if (x.arrivals) cudaFree(x.arrivals);
        if (x.part) cudaFree(x.part);
    }
    g_ws[dev].clear();
}

namespace {

// The plan of the line of these sequences for ctas CTAs, as the kernels make
// it: rows of 9 ints (attn_debug_packed_plan). in_order: what the starts say.
int plan_on_host(LineShape s, const std::vector<SeqLen> &seqs, bool in_order, int ctas, int max_ranges, int *out) {
    const int b = static_cast<int>(seqs.size());
    LineSum sum{0, 0, 0};
    for (const SeqLen &x : seqs) line_add(&sum, s, x.sq, x.sk, in_order);
    const LineDeal d = line_deal(&s, sum, ctas);
    auto find = [&](int at, int *before) {
        *before = 0;
        for (int i = 0; i < b; ++i) {
            const int sq = seqs[i].sq, sk = seqs[i].sk;
            const int cost = s.heads * line_before(s, sq, sk, line_units(s, sq, sk));
            if (at < *before + cost) return place_in_seq(s, i, sq, sk, at - *before);
            *before += cost;
        }
        return Place{b, 0, 0, 0};
    };
    int n = 0;
    for (int c = 0; c < d.parts; ++c) {
        int x0 = 0, unused = 0;
        const Place p = find(part_begin(d, c), &x0), e = find(part_begin(d, c + 1), &unused);
        if (p.seq >= b) continue;
        walk_part(s, b, p, e, seqs[p.seq], line_units(s, seqs[p.seq].sq, seqs[p.seq].sk), x0,
                  [&](int i) { return seqs[i]; },
                  [&](const UnitRange &r) {
                      if (n >= max_ranges) return false;
                      int first = c, cuts = 0;
                      for (int o = 0; r.slot >= 0 && o < d.parts; ++o)
                          if (part_cuts(s, d, o, r.x0, r.cost, r.steps) && cuts++ == 0) first = o - 1;
                      const int row[9] = {c, r.seq, r.head, r.unit, r.step0, r.nstep, r.slot, first, cuts + 1};
                      for (int i = 0; i < 9; ++i) out[9 * n + i] = row[i];
                      ++n;
                      return true;
                  });
    }
    return n;
}

bool plan_args_ok(const void *q, const void *k, const void *out, int b, int h, int h_kv, int ctas, int max_ranges) {
    return q && k && out && b >= 1 && h >= 1 && h_kv >= 1 && h % h_kv == 0 && h / h_kv <= 128 && ctas >= 1 &&
           max_ranges >= 1;
}

LineShape plan_shape(int h, int h_kv, int one_tile, int causal, int by_key, const LineBound &bound) {
    return by_key ? bwd_key_line(h_kv, h / h_kv, causal != 0, bound)
                  : pack_line(h_kv, h / h_kv, one_tile != 0, causal != 0, bound);
}

}  // namespace

extern "C" {

int attn_debug_packed_plan(const int *seqlens_q, const int *seqlens_k, int b, int h, int h_kv, int one_tile,
                           int causal, int by_key, int ctas, int max_ranges, int *out) try {
    if (!plan_args_ok(seqlens_q, seqlens_k, out, b, h, h_kv, ctas, max_ranges)) return -1;
    int64_t all_q = 0, all_k = 0;
    std::vector<SeqLen> seqs(b);
    for (int i = 0; i < b; ++i) {
        if (seqlens_q[i] < 0 || seqlens_k[i] < 0) return -1;
        seqs[i] = SeqLen{seqlens_q[i], seqlens_k[i]};
        all_q += seqlens_q[i];
        all_k += seqlens_k[i];
    }
    if (all_q > kMaxRows || all_k > kMaxRows) return -1;
    const LineBound bound{b, static_cast<int>(all_q), all_k, all_k};
    return plan_on_host(plan_shape(h, h_kv, one_tile, causal, by_key, bound), seqs, true, ctas, max_ranges, out);
} catch (...) {  // no exception leaves the library
    return -1;
}

int attn_debug_packed_starts(const int *cu_seqlens_q, const int *cu_seqlens_k, int b, int total_q, int total_k,
                             int h, int h_kv, int one_tile, int causal, int by_key, int ctas, int max_ranges,
                             int *out) try {
    if (!plan_args_ok(cu_seqlens_q, cu_seqlens_k, out, b, h, h_kv, ctas, max_ranges) || total_q < 1 || total_k < 1 ||
        total_q > kMaxRows || total_k > kMaxRows)
        return -1;
    std::vector<SeqLen> seqs(b);
    bool in_order = true;
    for (int i = 0; i < b; ++i) {
        int first = 0;
        in_order &= clamp_rows(cu_seqlens_q[i], cu_seqlens_q[i + 1], total_q, &first, &seqs[i].sq);
        in_order &= clamp_rows(cu_seqlens_k[i], cu_seqlens_k[i + 1], total_k, &first, &seqs[i].sk);
    }
    const LineBound bound{b, total_q, total_k, total_k};
    return plan_on_host(plan_shape(h, h_kv, one_tile, causal, by_key, bound), seqs, in_order, ctas, max_ranges, out);
} catch (...) {
    return -1;
}

int attn_debug_packed_shares(const int *seqlens_q, const int *seqlens_k, int b, int h, int h_kv, int causal,
                             int ctas, int *out) {
    if (!plan_args_ok(seqlens_q, seqlens_k, out, b, h, h_kv, ctas, 1) || ctas < 2) return -1;
    LineBound bound{b, 0, 0, 0};
    for (int i = 0; i < b; ++i) {
        if (seqlens_q[i] < 0 || seqlens_k[i] < 0 || seqlens_q[i] > kMaxRows - bound.total_q) return -1;
        bound.total_q += seqlens_q[i];
        bound.total_k += seqlens_k[i];
    }
    if (bound.total_k > kMaxRows) return -1;
    bound.max_k = bound.total_k;
    const LineShape q = bwd_query_line(h_kv, h / h_kv, causal != 0, bound),
                    kv = bwd_key_line(h_kv, h / h_kv, causal != 0, bound);
    LineSum qs{0, 0, 0}, kvs{0, 0, 0};
    for (int i = 0; i < b; ++i) {
        line_add(&qs, q, seqlens_q[i], seqlens_k[i], true);
        line_add(&kvs, kv, seqlens_q[i], seqlens_k[i], true);
    }
    out[0] = q.shift;
    out[1] = kv.shift;
    return key_ctas(q, qs, kv, kvs, ctas);
}

attn_status_t attn_fwd_packed(const void *q, const void *k, const void *v, const int32_t *cu_seqlens_q,
                              const int32_t *cu_seqlens_k, void *o, float *lse, int b, int total_q, int total_k,
                              int max_seqlen_q, int h, int h_kv, int d, int64_t q_stride, int64_t k_stride,
                              int64_t v_stride, float scale, int causal, attn_dtype_t dtype, cudaStream_t stream) {
    if (!q || !k || !v || !cu_seqlens_q || !cu_seqlens_k || !o || !lse) return ATTN_ERR_INVALID_ARG;
    if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(o, 16) || misaligned(lse, 4) ||
        misaligned(cu_seqlens_q, 4) || misaligned(cu_seqlens_k, 4))
        return ATTN_ERR_INVALID_ARG;
    if (total_k < 1) return ATTN_ERR_INVALID_ARG;
    attn_status_t st = check_packed(b, total_q, h, h_kv, d, scale, dtype);
    if (st == ATTN_OK && total_k > kMaxRows) st = ATTN_ERR_UNSUPPORTED;
    if (st == ATTN_OK) st = check_stride(q_stride, static_cast<int64_t>(h) * d);
    if (st == ATTN_OK) st = check_stride(k_stride, static_cast<int64_t>(h_kv) * d);
    if (st == ATTN_OK) st = check_stride(v_stride, static_cast<int64_t>(h_kv) * d);
    if (st != ATTN_OK) return st;
    int dev = 0, sms = 0;
    uint32_t *status = nullptr;
    if ((st = device_info(&dev, &status, &sms)) != ATTN_OK) return st;
    const bool bf16 = dtype == ATTN_BF16;
    PackArgs a;
    fill_pack(&a, o, lse, b, total_q, max_seqlen_q, h, h_kv, total_k, scale, causal != 0, status, sms);
    a.seqs.cu_q = cu_seqlens_q;
    a.seqs.cu_k = cu_seqlens_k;
    a.seqs.seqlens = nullptr;
    a.seqs.max_k = total_k;
    CUtensorMap tq, tk, tv;
    if (!encode_rows(&tq, q, bf16, d, h, h_kv, total_q, q_stride, a.tile_tokens) ||
        !encode_keys(&tk, k, bf16, d, h_kv, total_k, k_stride) ||
        !encode_keys(&tv, v, bf16, d, h_kv, total_k, v_stride))
        return ATTN_ERR_CUDA;
    return run_pack(&a, dev, d, stream, [&] { return launch_fwd_packed(d, bf16, tq, tk, tv, a, stream); });
}

attn_status_t attn_chunk_paged(const void *q, const void *k_pages, const void *v_pages, const int32_t *block_table,
                               const int32_t *cu_seqlens_q, const int32_t *seqlens_k, void *o, float *lse, int b,
                               int total_q, int max_seqlen_q, int h, int h_kv, int d, int num_pages, int page_size,
                               int max_pages_per_seq, int64_t q_stride, float scale, int causal,
                               attn_dtype_t dtype, cudaStream_t stream) {
    if (!q || !k_pages || !v_pages || !block_table || !cu_seqlens_q || !seqlens_k || !o || !lse)
        return ATTN_ERR_INVALID_ARG;
    if (misaligned(q, 16) || misaligned(k_pages, 16) || misaligned(v_pages, 16) || misaligned(o, 16) ||
        misaligned(lse, 4) || misaligned(block_table, 4) || misaligned(cu_seqlens_q, 4) || misaligned(seqlens_k, 4))
        return ATTN_ERR_INVALID_ARG;
    if (num_pages < 1 || page_size < 1 || max_pages_per_seq < 1) return ATTN_ERR_INVALID_ARG;
    attn_status_t st = check_packed(b, total_q, h, h_kv, d, scale, dtype);
    if (st == ATTN_OK) st = check_stride(q_stride, static_cast<int64_t>(h) * d);
    if (st != ATTN_OK) return st;
    // boxes of at most a page: page sizes are multiples of 16 keys
    if (page_size % 16 != 0) return ATTN_ERR_UNSUPPORTED;
    const int64_t max_k = static_cast<int64_t>(max_pages_per_seq) * page_size;
    if (max_k > kMaxRows) return ATTN_ERR_UNSUPPORTED;
    int dev = 0, sms = 0;
    uint32_t *status = nullptr;
    if ((st = device_info(&dev, &status, &sms)) != ATTN_OK) return st;
    const bool bf16 = dtype == ATTN_BF16;
    PackArgs a;
    fill_pack(&a, o, lse, b, total_q, max_seqlen_q, h, h_kv, max_k, scale, causal != 0, status, sms);
    a.seqs.cu_q = cu_seqlens_q;
    a.seqs.cu_k = nullptr;
    a.seqs.seqlens = seqlens_k;
    a.seqs.max_k = static_cast<int>(max_k);
    a.block_table = block_table;
    a.page_size = page_size;
    a.max_pages = max_pages_per_seq;
    a.num_pages = num_pages;
    a.box_rows = 128;  // the largest power of two that divides the page and the step
    while (page_size % a.box_rows != 0) a.box_rows /= 2;
    const int box0 = fwd_row_bytes(d) / 2;
    CUtensorMap tq, tk, tv;
    if (!encode_rows(&tq, q, bf16, d, h, h_kv, total_q, q_stride, a.tile_tokens) ||
        !encode_4d(&tk, k_pages, bf16, d, h_kv, page_size, num_pages, box0, a.box_rows, fwd_swizzle(d)) ||
        !encode_4d(&tv, v_pages, bf16, d, h_kv, page_size, num_pages, box0, a.box_rows, fwd_swizzle(d)))
        return ATTN_ERR_CUDA;
    return run_pack(&a, dev, d, stream, [&] { return launch_chunk_paged(d, bf16, tq, tk, tv, a, stream); });
}

attn_status_t attn_bwd_packed(const void *q, const void *k, const void *v, const void *o, const float *lse,
                              const void *dout, const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, void *dq,
                              void *dk, void *dv, int b, int total_q, int total_k, int h, int h_kv, int d,
                              int64_t q_stride, int64_t k_stride, int64_t v_stride, int64_t dq_stride,
                              int64_t dk_stride, int64_t dv_stride, float scale, int causal, attn_dtype_t dtype,
                              cudaStream_t stream) {
    for (const void *p : {q, k, v, o, dout, static_cast<const void *>(dq), static_cast<const void *>(dk),
                          static_cast<const void *>(dv)})
        if (!p || misaligned(p, 16)) return ATTN_ERR_INVALID_ARG;
    for (const void *p : {static_cast<const void *>(lse), static_cast<const void *>(cu_seqlens_q),
                          static_cast<const void *>(cu_seqlens_k)})
        if (!p || misaligned(p, 4)) return ATTN_ERR_INVALID_ARG;
    if (total_k < 1) return ATTN_ERR_INVALID_ARG;
    attn_status_t st = check_packed(b, total_q, h, h_kv, d, scale, dtype);
    if (st == ATTN_OK && total_k > kMaxRows) st = ATTN_ERR_UNSUPPORTED;
    if (st == ATTN_OK) st = check_units(b, total_k, 128, h_kv);
    const int64_t qrow = static_cast<int64_t>(h) * d, krow = static_cast<int64_t>(h_kv) * d;
    for (int64_t s : {q_stride, dq_stride})
        if (st == ATTN_OK) st = check_stride(s, qrow);
    for (int64_t s : {k_stride, v_stride, dk_stride, dv_stride})
        if (st == ATTN_OK) st = check_stride(s, krow);
    if (st != ATTN_OK) return st;
    int dev = 0, sms = 0;
    uint32_t *status = nullptr;
    if ((st = device_info(&dev, &status, &sms)) != ATTN_OK) return st;
    if (sms < 2) return ATTN_ERR_UNSUPPORTED;
    const bool bf16 = dtype == ATTN_BF16;
    PackBwdArgs a;
    a.seqs.cu_q = cu_seqlens_q;
    a.seqs.cu_k = cu_seqlens_k;
    a.seqs.seqlens = nullptr;
    a.seqs.b = b;
    a.seqs.total_q = total_q;
    a.seqs.max_k = total_k;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.o = o;
    a.dout = dout;
    a.lse = lse;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.dq_stride = dq_stride;
    a.dk_stride = dk_stride;
    a.dv_stride = dv_stride;
    a.h = h;
    a.group = h / h_kv;
    a.tile_tokens = pack_tile_tokens(a.group);
    a.total_q = total_q;
    a.causal = causal ? 1 : 0;
    a.scale = scale;
    a.scale_log2 = scale * kLog2e;
    a.status = status;
    a.flags = debug_flags();
    a.group_inv = pack_group_inv(a.group);
    fast_division(a.group, &a.group_mul, &a.group_div);
    const LineBound bound{b, total_q, total_k, total_k};
    a.line[0] = bwd_query_line(h_kv, a.group, causal != 0, bound);
    a.line[1] = bwd_key_line(h_kv, a.group, causal != 0, bound);
    a.ctas = sms;
    CUtensorMap tq, tk, tv, tdo;
    if (!encode_rows(&tq, q, bf16, d, h, h_kv, total_q, q_stride, a.tile_tokens) ||
        !encode_rows(&tdo, dout, bf16, d, h, h_kv, total_q, qrow, a.tile_tokens) ||
        !encode_keys(&tk, k, bf16, d, h_kv, total_k, k_stride) ||
        !encode_keys(&tv, v, bf16, d, h_kv, total_k, v_stride))
        return ATTN_ERR_CUDA;
    const size_t tile = 128 * static_cast<size_t>(d) * sizeof(float);
    const size_t part_q = 2 * a.ctas * tile, part_kv = 4 * a.ctas * tile;
    const size_t ld = static_cast<size_t>(total_q) * h * sizeof(float2);
    Workspace w;
    if ((st = get_workspace(dev, stream, 2 * sms, part_q + part_kv + ld, &w)) != ATTN_OK) return st;
    a.arrivals = w.arrivals;
    a.call = w.call;
    a.part[0] = reinterpret_cast<float *>(w.part);
    a.part[1] = reinterpret_cast<float *>(w.part + part_q);
    a.ld = reinterpret_cast<float2 *>(w.part + part_q + part_kv);
    const cudaError_t e = launch_bwd_packed(d, bf16, tq, tk, tv, tdo, a, stream);
    const cudaError_t ef = w.owned ? cudaFreeAsync(w.owned, stream) : cudaSuccess;
    return (e == cudaSuccess && ef == cudaSuccess) ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t attn_paged_plan(const int32_t *seqlens_k, const int32_t *new_lens, int32_t *block_table,
                              const int32_t *free_pages, const int32_t *free_count, int32_t *cu_seqlens_q,
                              int32_t *seqlens_out, int64_t *slot_map, int32_t *free_left, int b,
                              int max_pages_per_seq, int page_size, int num_free, int64_t max_tokens,
                              cudaStream_t stream) {
    if (!seqlens_k || !new_lens || !block_table || !free_pages || !free_count || !cu_seqlens_q || !seqlens_out ||
        !slot_map || !free_left)
        return ATTN_ERR_INVALID_ARG;
    for (const void *p : {static_cast<const void *>(seqlens_k), static_cast<const void *>(new_lens),
                          static_cast<const void *>(block_table), static_cast<const void *>(free_pages),
                          static_cast<const void *>(free_count), static_cast<const void *>(cu_seqlens_q),
                          static_cast<const void *>(seqlens_out), static_cast<const void *>(free_left)})
        if (misaligned(p, 4)) return ATTN_ERR_INVALID_ARG;
    if (misaligned(slot_map, 8)) return ATTN_ERR_INVALID_ARG;
    if (b < 1 || max_pages_per_seq < 1 || page_size < 1 || num_free < 1 || max_tokens < 1)
        return ATTN_ERR_INVALID_ARG;
    if (b > 65535 || static_cast<int64_t>(max_pages_per_seq) * page_size > 0x7fffffffLL ||
        max_tokens > 0x7fffffffLL)
        return ATTN_ERR_UNSUPPORTED;
    // every block reads all inputs while others write outputs
    const size_t n4 = static_cast<size_t>(b) * 4;
    const struct {
        const void *p;
        size_t n;
    } in[4] = {{seqlens_k, n4}, {new_lens, n4}, {free_pages, static_cast<size_t>(num_free) * 4}, {free_count, 4}},
      out[5] = {{block_table, n4 * max_pages_per_seq},
                {cu_seqlens_q, n4 + 4},
                {seqlens_out, n4},
                {slot_map, static_cast<size_t>(max_tokens) * 8},
                {free_left, 4}};
    for (int i = 0; i < 5; ++i) {
        for (const auto &x : in)
            if (overlap(out[i].p, out[i].n, x.p, x.n)) return ATTN_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return ATTN_ERR_INVALID_ARG;
    }
    int dev = 0, sms = 0;
    uint32_t *status = nullptr;
    const attn_status_t st = device_info(&dev, &status, &sms);
    if (st != ATTN_OK) return st;
    PlanArgs a;
    a.seqlens = seqlens_k;
    a.new_lens = new_lens;
    a.block_table = block_table;
    a.free_pages = free_pages;
    a.free_count = free_count;
    a.cu_seqlens_q = cu_seqlens_q;
    a.seqlens_out = seqlens_out;
    a.slot_map = slot_map;
    a.free_left = free_left;
    a.b = b;
    a.max_pages = max_pages_per_seq;
    a.page_size = page_size;
    a.num_free = num_free;
    a.max_tokens = max_tokens;
    return launch_paged_plan(a, sms, stream) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t attn_paged_write(const void *k, const void *v, const int64_t *slot_map, void *k_pages, void *v_pages,
                               int64_t tokens, int h_kv, int d, int num_pages, int page_size, int64_t k_stride,
                               int64_t v_stride, attn_dtype_t dtype, cudaStream_t stream) {
    if (!k || !v || !slot_map || !k_pages || !v_pages) return ATTN_ERR_INVALID_ARG;
    if (misaligned(k, 16) || misaligned(v, 16) || misaligned(k_pages, 16) || misaligned(v_pages, 16) ||
        misaligned(slot_map, 8))
        return ATTN_ERR_INVALID_ARG;
    if (tokens < 1 || h_kv < 1 || num_pages < 1 || page_size < 1) return ATTN_ERR_INVALID_ARG;
    if (dtype != ATTN_FP16 && dtype != ATTN_BF16) return ATTN_ERR_INVALID_ARG;
    if (d != 16 && d != 32 && d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
    if (h_kv > 65535 || tokens > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
    const int64_t row = static_cast<int64_t>(h_kv) * d;
    attn_status_t st = check_stride(k_stride, row);
    if (st == ATTN_OK) st = check_stride(v_stride, row);
    if (st != ATTN_OK) return st;
    int dev = 0, sms = 0;
    uint32_t *status = nullptr;
    if ((st = device_info(&dev, &status, &sms)) != ATTN_OK) return st;
    WriteArgs a;
    a.k = static_cast<const uint4 *>(k);
    a.v = static_cast<const uint4 *>(v);
    a.slot_map = slot_map;
    a.k_pages = static_cast<uint4 *>(k_pages);
    a.v_pages = static_cast<uint4 *>(v_pages);
    a.tokens = tokens;
    a.words = static_cast<int>(row / 8);
    a.k_stride = k_stride / 8;
    a.v_stride = v_stride / 8;
    a.slots = static_cast<int64_t>(num_pages) * page_size;
    if (a.tokens * a.words > (1ll << 40)) return ATTN_ERR_UNSUPPORTED;
    return launch_paged_write(a, stream) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // extern "C"
