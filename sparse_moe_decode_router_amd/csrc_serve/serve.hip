// serve.hip - host side of attention, the cache's upkeep and the 4-bit products:
// argument checks, launch rules and their part of the C ABI declared in
// include/moe_serve.h.
#include "serve_host.h"

#include "attn_decode.h"
#include "attn_prompt.h"
#include "kv_pages.h"
#include "w4_linear.h"

using namespace moe::serve;

namespace {

constexpr int kMaxW4Tokens = 1 << 21;              // of one launch: 2^15 times 64

// Row tiles as workgroups, split over the keys where there are few of them.
// With more of them than fit at once, long and short ones would leave the chip
// part empty in the end (8192 tokens, window 4096, 14 heads: 18% of their time):
// then every workgroup takes an equal share of all tiles of keys.
struct PromptPlan {
    int64_t tiles;
    int split, units;
    int64_t slots;  // of partial results
};
// Partial results of a call that splits row tiles, for each workgroup that the
// chip holds at once: bounds the workspace (512 such workgroups, head_dim 128: 136
// MB), and the work of joining where many sequences have few new tokens (3 parts
// against 8, 64 sequences of up to 4 new ones of 4096, 56 heads on 8: 155 and 195
// us; 4 against 9, 16 of up to 3 of 32768: 295 and 331).
constexpr int kPromptPartsPerSlot = 4;

// Parts of a row tile, where `row_tiles` of them per kv head are sure to be full.
int64_t prompt_parts(const moe_kv_cache &kv, const moe_attn_config &c, int64_t row_tiles) {
    const int64_t sure = std::max<int64_t>(1, row_tiles) * kv.kv_heads;
    // T tiles of keys in P parts take about T / P rounds and as many again as P to
    // join them: the square root of T parts, and four tiles in each at least
    // (300 tokens of 8192, 14 heads: 8, 10 and 15 parts 46, 48 and 58 us; 100 of
    // 2100, 4 heads: 2, 4 and 8 parts 33, 24 and 21 us).
    int64_t keys = c.longest;
    if (c.window > 0) keys = std::min<int64_t>(keys, (int64_t)c.window + c.sinks + kPromptRows);
    const int64_t tiles = (keys + kPromptKeys - 1) / kPromptKeys;
    int64_t parts = 1;
    while (parts < 64 && parts * parts < tiles) ++parts;
    return std::min<int64_t>({prompt_slots(kv.head_dim) / sure, parts, tiles / 4});
}
// The plan for `row_tiles` full row tiles per kv head and at most `more` part-filled
// ones beside them.
PromptPlan prompt_plan_of(const moe_kv_cache &kv, const moe_attn_config &c, int64_t row_tiles,
                          int64_t more) {
    PromptPlan p;
    p.tiles = row_tiles + more;
    const int slots = prompt_slots(kv.head_dim);
    const int64_t most = (int64_t)slots * kPromptPartsPerSlot;
    p.split = (int)std::max<int64_t>(
        1, std::min(prompt_parts(kv, c, row_tiles),
                    most / std::max<int64_t>(1, p.tiles * kv.kv_heads)));
    p.units = std::max<int64_t>(1, row_tiles) * kv.kv_heads > slots
                  ? std::max(1, slots / kv.kv_heads)
                  : 0;
    p.slots = p.units ? 2 * (int64_t)p.units : p.split > 1 ? p.tiles * p.split : 0;
    p.slots *= kv.kv_heads;
    return p;
}
int64_t full_row_tiles(const moe_kv_cache &kv, const moe_attn_config &c, int64_t tokens) {
    return tokens * (c.q_heads / kv.kv_heads) / kPromptRows;
}
PromptPlan prompt_plan(const moe_kv_cache &kv, const moe_attn_config &c, int tokens, int batch) {
    return prompt_plan_of(kv, c, full_row_tiles(kv, c, tokens), std::min(batch, tokens));
}
// Slots that no call of up to `tokens` tokens goes beyond: fewer row tiles are
// split more finely, so the largest call need not be the one that takes most.
// (A call has as many part-filled row tiles as sequences or fewer, and with r full
// row tiles no more tokens than those and one more would hold.)
int64_t prompt_slots_up_to(const moe_kv_cache &kv, const moe_attn_config &c, int tokens) {
    const int64_t last = full_row_tiles(kv, c, tokens), group = c.q_heads / kv.kv_heads;
    const int slots = prompt_slots(kv.head_dim);
    int64_t most = 0;
    // (From slots + 1 full row tiles on, all take equal shares.)
    for (int64_t r = 0; r <= std::min<int64_t>(last, slots + 1); ++r) {
        const int64_t more = std::min<int64_t>(
            {c.batch, tokens, ((r + 1) * kPromptRows - 1) / group});
        const PromptPlan p = prompt_plan_of(kv, c, r, 0);
        const int64_t parts = prompt_parts(kv, c, r);   // before it is bounded
        if (p.units)
            most = std::max(most, p.slots);
        else if (parts > 1)
            most = std::max(most, std::min((r + more) * parts * kv.kv_heads,
                                           (int64_t)slots * kPromptPartsPerSlot));
    }
    return most;
}

template <class F>
moe_status with_group(int group, bool z, F f) {
    auto g = [&](auto gl) { return z ? f(gl, std::true_type()) : f(gl, std::false_type()); };
    if (group == 32) return g(std::integral_constant<int, 5>());
    if (group == 64) return g(std::integral_constant<int, 6>());
    return g(std::integral_constant<int, 7>());
}
// The fewest rows per workgroup that leave no compute unit two workgroups: a
// second one on some of them costs more than larger tiles do, and from there
// on larger tiles spread x over more rows.  Measured with 7168 columns, bf16, zero
// points, in us of device time:
//   weight rows            4096  4111  6144  8192  9216 12288 18432 36864
//    8 tokens, 16 rows      6.9   8.8  10.2  11.9  15.9  19.0  27.7  49.9
//              32           9.0   9.1   9.2   9.8  14.4  16.6  24.5  40.1
//              64          12.9  12.9  13.1  13.5  14.4  15.9  27.2  40.8
//   16 tokens, 16           7.9  11.0  12.0  14.6  20.0  23.3  35.5  63.4
//              32           9.9  10.0  10.1  11.0  17.6  20.0  28.5  46.7
//              64          14.0  14.1  14.3  15.6  16.4  17.9  29.7  44.8
//   32 tokens, 16          11.3  18.8  19.9  22.2  31.7  36.6  57.8 105.2
//              64          15.9  15.9  16.1  19.2  20.8  22.1  40.1  61.9
//   64 tokens, 16          17.3  28.4  30.2  34.1  47.4  53.7  84.2 155.5
//              32          19.6  19.7  20.4  24.4  41.0  44.2  64.9 108.9
//              64          30.6  30.7  30.9  32.3  33.0  33.9  64.4  96.3
// (A form of 32 rows for 17 to 32 tokens, which there is not, would take 11.7 to
// 15.2 from 4111 to 8192 rows.)  A single token has next to no x to spread: 8
// waves of four steps ahead against 4 of two, 1152 rows 5.2 and 6.6, 4096 6.1 and
// 7.0, 4111 7.7 and 7.9, 9216 12.4 and 11.6, 36864 39.7 and 37.7.
template <class T, int GL, bool Z>
moe_status w4_launch(const W4Args &a, int cus, hipStream_t stream) {
    auto go = [&](auto kernel, int nt, int rt, int w) {
        const dim3 grid((a.n + 16 * rt - 1) / (16 * rt), (a.tokens + 16 * nt - 1) / (16 * nt));
        kernel<<<grid, 64 * w, 0, stream>>>(a);
        return launched();
    };
    const int rt = a.n <= 16 * cus ? 1 : a.n <= 32 * cus ? 2 : 4;
    if (a.tokens <= 4)
        return rt == 1 ? go(k_w4<T, 1, 1, 1, 8, 4, GL, Z>, 1, 1, 8)
                       : go(k_w4<T, 1, 1, 1, 4, 2, GL, Z>, 1, 1, 4);
    if (a.tokens <= 8)
        return rt == 1   ? go(k_w4<T, 1, 2, 1, 8, 2, GL, Z>, 1, 1, 8)
               : rt == 2 ? go(k_w4<T, 1, 2, 2, 4, 2, GL, Z>, 1, 2, 4)
                         : go(k_w4<T, 1, 2, 4, 4, 2, GL, Z>, 1, 4, 4);
    if (a.tokens <= 16)
        return rt == 1   ? go(k_w4<T, 1, 4, 1, 8, 2, GL, Z>, 1, 1, 8)
               : rt == 2 ? go(k_w4<T, 1, 4, 2, 4, 2, GL, Z>, 1, 2, 4)
                         : go(k_w4<T, 1, 4, 4, 4, 2, GL, Z>, 1, 4, 4);
    if (a.tokens <= 32)
        return rt == 1 ? go(k_w4<T, 2, 8, 1, 8, 2, GL, Z>, 2, 1, 8)
                       : go(k_w4<T, 2, 8, 4, 8, 1, GL, Z>, 2, 4, 8);
    return rt == 1   ? go(k_w4<T, 4, 16, 1, 8, 1, GL, Z>, 4, 1, 8)
           : rt == 2 ? go(k_w4<T, 4, 16, 2, 8, 1, GL, Z>, 4, 2, 8)
                     : go(k_w4<T, 4, 16, 4, 4, 1, GL, Z>, 4, 4, 4);
}

PagesArgs pages_args(const moe_kv_cache &kv, int n, void *scratch) {
    PagesArgs a = {};
    a.tables = kv.tables;
    a.lengths = kv.lengths;
    a.refs = kv.refs;
    a.flags = kv.flags;
    a.scratch = (int32_t *)scratch;
    a.n = n;
    a.pages = kv.pages;
    a.page_log2 = log2_of(kv.page);
    a.seqs = kv.seqs;
    a.cols = kv.cols;
    return a;
}
MoveArgs move_args(const moe_kv_cache &kv) {
    MoveArgs m = {};
    m.data = (char *)kv.data;
    m.plane_bytes = plane_bytes(kv);
    m.page_bytes = m.plane_bytes / kv.pages;
    m.planes = 2 * kv.layers;
    m.pages = kv.pages;
    return m;
}

}  // namespace

extern "C" {

int32_t moe_serve_last_hip_error(void) { return g_last_hip; }

moe_status moe_kv_validate(const moe_kv_cache *kv) {
    if (!kv || !kv->data || !kv->tables || !kv->lengths || !kv->refs || !kv->flags)
        return MOE_ERR_INVALID_ARG;
    if (kv->layers < 1 || kv->pages < 1 || kv->kv_heads < 1 || kv->seqs < 1 || kv->cols < 1)
        return MOE_ERR_INVALID_ARG;
    if (kv->dtype < MOE_BF16 || kv->dtype > MOE_E4M3) return MOE_ERR_INVALID_ARG;
    if (kv->dtype != MOE_E4M3 && (kv->k_scale || kv->v_scale)) return MOE_ERR_INVALID_ARG;
    if (!aligned(kv->data, 16)) return MOE_ERR_INVALID_ARG;
    if (kv->page < 16 || kv->page > 1024 || (kv->page & (kv->page - 1))) return MOE_ERR_UNSUPPORTED;
    if (kv->seqs > kMaxRows || kv->kv_heads > 1024 || kv->layers > 4096) return MOE_ERR_UNSUPPORTED;
    if ((int64_t)kv->cols * kv->page >= (1ll << 31) - 2048 ||
        (int64_t)kv->seqs * kv->cols >= (1ll << 31) / (kv->page / 16))
        return MOE_ERR_UNSUPPORTED;
    return with_dim(kv->head_dim, [](auto) { return MOE_OK; });
}

moe_status moe_kv_append(const moe_kv_cache *kv, int32_t layer, const void *k, const void *v,
                         int32_t dtype, int64_t token_stride, int64_t head_stride, int32_t tokens,
                         const int32_t *cu, int32_t batch, moe_stream_t stream) {
    return moe_kv_append_granted(kv, layer, k, v, dtype, token_stride, head_stride, tokens, cu,
                                 batch, nullptr, stream);
}

moe_status moe_kv_append_granted(const moe_kv_cache *kv, int32_t layer, const void *k,
                                 const void *v, int32_t dtype, int64_t token_stride,
                                 int64_t head_stride, int32_t tokens, const int32_t *cu,
                                 int32_t batch, const int32_t *granted, moe_stream_t stream) {
    moe_status s = moe_kv_validate(kv);
    if (s != MOE_OK) return s;
    if (layer < 0 || layer >= kv->layers || tokens < 0 || batch < 0 || batch > kv->seqs ||
        tokens > kMaxRows)
        return MOE_ERR_INVALID_ARG;
    if (!cu && tokens != batch) return MOE_ERR_INVALID_ARG;
    if (tokens == 0 || batch == 0) return MOE_OK;
    if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return MOE_ERR_INVALID_ARG;
    if ((s = check_types(*kv, dtype)) != MOE_OK) return s;
    if ((s = check_strides(token_stride, head_stride, kv->kv_heads, kv->head_dim)) != MOE_OK)
        return s;
    int cus;
    if ((s = compute_units(&cus)) != MOE_OK) return s;
    AppendArgs a = {};
    a.k = k;
    a.v = v;
    a.kc = plane(*kv, layer, 0);
    a.vc = plane(*kv, layer, 1);
    a.tables = kv->tables;
    a.lengths = kv->lengths;
    a.cu = cu;
    a.granted = granted;
    a.k_scale = kv->k_scale;
    a.v_scale = kv->v_scale;
    a.token_stride = token_stride;
    a.head_stride = head_stride;
    a.tokens = tokens;
    a.batch = batch;
    a.pages = kv->pages;
    a.cols = kv->cols;
    a.page_log2 = log2_of(kv->page);
    a.kv_heads = kv->kv_heads;
    a.head_dim = kv->head_dim;
    // Two rounds of the workgroup's threads, where there are tokens enough to
    // fill the chip that way.
    const int per_token = kv->kv_heads * kv->head_dim / 8;
    a.per_block = std::max(1 + (tokens >> 23), std::min(512 / per_token, tokens / (4 * cus)));
    const int grid = (tokens + a.per_block - 1) / a.per_block;
    return with_types(dtype, kv->dtype == MOE_E4M3, [&](auto t, auto f8) {
        k_kv_append<decltype(t), decltype(f8)::value><<<grid, 256, 0, stream>>>(a);
        return launched();
    });
}

size_t moe_kv_scratch_size(const moe_kv_cache *kv, int32_t n) {
    if (moe_kv_validate(kv) != MOE_OK || n < 0 || n > kMaxRows) return 0;
    return sizeof(int32_t) *
           (kScratchHead + std::max<size_t>(3 * (size_t)kv->pages, 3 * (size_t)n + kv->pages));
}

moe_status moe_kv_free(const moe_kv_cache *kv, const int32_t *seqs, int32_t n,
                       moe_stream_t stream) {
    moe_status s = moe_kv_validate(kv);
    if (s != MOE_OK) return s;
    if (n < 0 || n > kv->seqs) return MOE_ERR_INVALID_ARG;
    if (n == 0) return MOE_OK;
    if (!seqs) return MOE_ERR_INVALID_ARG;
    PagesArgs a = pages_args(*kv, n, nullptr);
    a.from = seqs;
    k_kv_free<<<std::min(n, 1 << 20), 256, 0, stream>>>(a);
    return launched();
}

moe_status moe_kv_fork(const moe_kv_cache *kv, const int32_t *parents, const int32_t *children,
                       int32_t n, void *scratch, moe_stream_t stream) {
    moe_status s = moe_kv_validate(kv);
    if (s != MOE_OK) return s;
    if (n < 0 || n > kv->seqs) return MOE_ERR_INVALID_ARG;
    if (n == 0) return MOE_OK;
    if (!parents || !children) return MOE_ERR_INVALID_ARG;
    if (!scratch || !aligned(scratch, 16)) return MOE_ERR_WORKSPACE;
    PagesArgs a = pages_args(*kv, n, scratch);
    a.from = parents;
    a.to = children;
    k_kv_fork<<<1, kPagesThreads, 0, stream>>>(a);
    if ((s = launched()) != MOE_OK) return s;
    MoveArgs m = move_args(*kv);
    m.n = n;
    m.from = a.scratch + kScratchHead;
    m.to = m.from + 1;
    m.stride = 2;
    const int64_t items = (int64_t)n * m.planes * ((m.page_bytes + kMoveChunk - 1) / kMoveChunk);
    k_kv_move<<<(int)std::min<int64_t>(items, 2048), 256, 0, stream>>>(m);
    return launched();
}

moe_status moe_kv_extend(const moe_kv_cache *kv, const int32_t *seqs, const int32_t *counts,
                         int32_t n, void *scratch, moe_stream_t stream) {
    return moe_kv_extend_granted(kv, seqs, counts, n, nullptr, scratch, stream);
}

moe_status moe_kv_extend_granted(const moe_kv_cache *kv, const int32_t *seqs,
                                 const int32_t *counts, int32_t n, int32_t *granted,
                                 void *scratch, moe_stream_t stream) {
    moe_status s = moe_kv_validate(kv);
    if (s != MOE_OK) return s;
    if (n < 0 || n > kv->seqs) return MOE_ERR_INVALID_ARG;
    if (n == 0) return MOE_OK;
    if (!counts) return MOE_ERR_INVALID_ARG;
    if (!scratch || !aligned(scratch, 16)) return MOE_ERR_WORKSPACE;
    PagesArgs a = pages_args(*kv, n, scratch);
    a.from = seqs;
    a.counts = counts;
    a.granted = granted;
    k_kv_extend<<<1, kPagesThreads, 0, stream>>>(a);
    return launched();
}

moe_status moe_kv_compact(const moe_kv_cache *kv, int32_t *new_tables, int32_t *new_refs,
                          void *scratch, moe_stream_t stream) {
    moe_status s = moe_kv_validate(kv);
    if (s != MOE_OK) return s;
    if (!new_tables || !new_refs) return MOE_ERR_INVALID_ARG;
    if (!scratch || !aligned(scratch, 16)) return MOE_ERR_WORKSPACE;
    PagesArgs a = pages_args(*kv, 0, scratch);
    a.new_tables = new_tables;
    a.new_refs = new_refs;
    k_kv_compact<<<1, kPagesThreads, 0, stream>>>(a);
    if ((s = launched()) != MOE_OK) return s;
    MoveArgs m = move_args(*kv);
    m.count = a.scratch;
    m.n = kv->pages / 2;
    m.to = a.scratch + kScratchHead;
    m.from = m.to + kv->pages;
    m.place = m.from + kv->pages;
    m.stride = 1;
    m.tables = kv->tables;
    m.new_tables = new_tables;
    m.entries = (int64_t)kv->seqs * kv->cols;
    k_kv_move<<<2048, 256, 0, stream>>>(m);
    return launched();
}

moe_status moe_attn_validate(const moe_kv_cache *kv, const moe_attn_config *c) {
    const moe_status s = moe_kv_validate(kv);
    if (s != MOE_OK) return s;
    if (!c || c->q_heads < 1 || c->q_heads % kv->kv_heads || c->batch < 1 || c->batch > kv->seqs ||
        c->longest < 1 || c->window < 0 || c->sinks < 0 || !(c->scale > 0.f) ||
        !(c->scale < 1e30f))
        return MOE_ERR_INVALID_ARG;
    if (c->q_heads / kv->kv_heads > 1024) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

moe_status moe_attn_workspace(const moe_kv_cache *kv, const moe_attn_config *c, int32_t tokens,
                              size_t *workspace, size_t *counters) {
    const moe_status s = moe_attn_validate(kv, c);
    if (s != MOE_OK) return s;
    if (!workspace || !counters || tokens < 0 || tokens > kMaxRows) return MOE_ERR_INVALID_ARG;
    if (tokens == 0) {
        const int hg = (c->q_heads / kv->kv_heads + 15) / 16;
        const size_t heads = (size_t)kv->kv_heads * hg;
        *workspace = sizeof(float) * 16 * (kv->head_dim + 2) * heads *
                     ((size_t)decode_split(*kv, *c, c->longest) + c->batch);
        *counters = sizeof(uint32_t) * heads * c->batch;
    } else {
        const PromptPlan p = prompt_plan(*kv, *c, tokens, c->batch);
        *workspace = sizeof(float) * kPromptRows * (kv->head_dim + 2) *
                     (size_t)prompt_slots_up_to(*kv, *c, tokens);
        *counters = sizeof(uint32_t) * (size_t)p.tiles * kv->kv_heads;
    }
    return MOE_OK;
}

moe_status moe_attn_decode(const moe_kv_cache *kv, const moe_attn_config *c, int32_t layer,
                           const void *q, int32_t dtype, int64_t token_stride, int64_t head_stride,
                           int32_t batch, void *out, float *lse, void *workspace, uint32_t *counters,
                           moe_stream_t stream) {
    moe_status s = check_attn(kv, c, layer, q, dtype, token_stride, head_stride, batch, out, lse,
                              workspace, counters);
    if (s != MOE_OK) return s;
    if (!workspace || !counters) return MOE_ERR_WORKSPACE;
    AttnArgs a = attn_args(*kv, *c, layer);
    a.split = decode_split(*kv, *c, c->longest);
    const int64_t grid = ((int64_t)a.split + batch) * a.kv_heads * a.head_groups;
    if (grid > kMaxGrid256) return MOE_ERR_UNSUPPORTED;
    int cus;
    if ((s = compute_units(&cus)) != MOE_OK) return s;
    a.q = q;
    a.q_token = token_stride;
    a.q_head = head_stride;
    a.out = out;
    a.lse = lse;
    a.part = (float *)workspace;
    a.counters = counters;
    a.batch = batch;
    return with_types(dtype, kv->dtype == MOE_E4M3, [&](auto t, auto f8) {
        return with_dim(kv->head_dim, [&](auto d) {
            k_attn_decode<decltype(t), decltype(f8)::value, decltype(d)::value>
                <<<(int)grid, kDecodeThreads, 0, stream>>>(a);
            return launched();
        });
    });
}

moe_status moe_attn_prompt(const moe_kv_cache *kv, const moe_attn_config *c, int32_t layer,
                           const void *q, int32_t dtype, int64_t token_stride, int64_t head_stride,
                           int32_t tokens, const int32_t *cu, int32_t batch, void *out, float *lse,
                           void *workspace, uint32_t *counters, moe_stream_t stream) {
    if (tokens == 0 && moe_attn_validate(kv, c) == MOE_OK) return MOE_OK;
    moe_status s = check_attn(kv, c, layer, q, dtype, token_stride, head_stride, batch, out, lse,
                              workspace, counters);
    if (s != MOE_OK) return s;
    if (!cu || tokens < 0 || tokens > kMaxRows) return MOE_ERR_INVALID_ARG;
    int cus;
    if ((s = compute_units(&cus)) != MOE_OK) return s;
    AttnArgs a = attn_args(*kv, *c, layer);
    a.q = q;
    a.q_token = token_stride;
    a.q_head = head_stride;
    a.cu = cu;
    a.out = out;
    a.lse = lse;
    a.part = (float *)workspace;
    a.counters = counters;
    a.batch = batch;
    a.tokens = tokens;
    const PromptPlan p = prompt_plan(*kv, *c, tokens, batch);
    a.split = p.split;
    a.units = p.units;
    a.row_tiles = (int32_t)std::min<int64_t>(p.tiles, 0x7FFFFFFF);
    if (p.slots && (!workspace || !counters)) return MOE_ERR_WORKSPACE;
    const int64_t grid = kv->kv_heads * (p.units ? p.units : p.tiles * p.split);
    if (grid > kMaxGrid256) return MOE_ERR_UNSUPPORTED;
    return with_types(dtype, kv->dtype == MOE_E4M3, [&](auto t, auto f8) {
        return with_dim(kv->head_dim, [&](auto d) {
            k_attn_prompt<decltype(t), decltype(f8)::value, decltype(d)::value>
                <<<(int)grid, kPromptThreads, 0, stream>>>(a);
            return launched();
        });
    });
}

moe_status moe_w4_linear(const void *x, int64_t x_stride, int32_t dtype, const uint8_t *codes,
                         const void *scales, const uint8_t *zeros, int32_t tokens, int32_t k,
                         int32_t n, int32_t group, void *y, moe_stream_t stream) {
    if ((dtype != MOE_BF16 && dtype != MOE_FP16) || !codes || !scales || tokens < 0 || k < 1 ||
        n < 1 || tokens > kMaxRows)
        return MOE_ERR_INVALID_ARG;
    if (group != 32 && group != 64 && group != 128) return MOE_ERR_UNSUPPORTED;
    if (k % group || k > 1 << 24 || n > 1 << 24 || x_stride > 1 << 25) return MOE_ERR_UNSUPPORTED;
    if (tokens == 0) return MOE_OK;
    if (!x || !y || x_stride < 0 || x_stride % 8 || !aligned(x, 16) || !aligned(codes, 16))
        return MOE_ERR_INVALID_ARG;
    int cus;
    moe_status s = compute_units(&cus);
    if (s != MOE_OK) return s;
    W4Args a = {};
    a.scales = (const uint16_t *)scales;
    a.codes = codes;
    a.zeros = zeros;
    a.x_stride = x_stride;
    a.k = k;
    a.n = n;
    for (int64_t t = 0; t < tokens && s == MOE_OK; t += kMaxW4Tokens) {
        a.x = (const uint16_t *)x + t * x_stride;
        a.y = (uint16_t *)y + t * n;
        a.tokens = (int32_t)std::min<int64_t>(tokens - t, kMaxW4Tokens);
        s = with_types(dtype, false, [&](auto ty, auto) {
            return with_group(group, zeros != nullptr, [&](auto gl, auto z) {
                return w4_launch<decltype(ty), decltype(gl)::value, decltype(z)::value>(a, cus,
                                                                                        stream);
            });
        });
    }
    return s;
}

}  // extern "C"
