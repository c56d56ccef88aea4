// generate.hip - host side of the rotated append and of sampling: argument checks,
// launch rules and their part of the C ABI declared in include/moe_serve.h.
#include "serve_host.h"

#include "kv_rotary.h"
#include "sample.h"

using namespace moe::serve;

namespace {

constexpr int kMaxVocab = 1 << 19;     // counts of 20 bits, weights of 44 in one integer
// Workgroups that a sampling call's launches aim at: two for each compute unit.  Every
// one has a chain of latencies of its own (64 rows of 163840 in f32, 512 rows of 100003 in
// bf16, us: 512 for both launches 66 and 152, 1024 for the second 79 and 160, for both
// 76 and 182, 512 and 2048 100 and 187).
constexpr int kSampleGrid = 512;

constexpr int logits_per_chunk(int dtype) { return dtype == MOE_F32 ? 4 : 8; }
// 16-byte chunks of a row, wherever it begins.
constexpr int row_chunks(int vocab, int dtype) {
    const int per = logits_per_chunk(dtype);
    return (vocab + per - 1) / per + 1;
}
// The fewest slices whose lanes have at most kSampleChunks chunks.
constexpr int least_slices(int vocab, int dtype) {
    const int most = kSampleWaves * 64 * kSampleChunks;
    return (row_chunks(vocab, dtype) + most - 1) / most;
}
static_assert(least_slices(kMaxVocab, MOE_F32) <= kSampleMaxSlices, "slices of the largest row");
// Slices of a row, at most `most`.
int sample_slices(int rows, int vocab, int dtype, int most) {
    // No wave has less than one chunk a lane.
    const int useful = (row_chunks(vocab, dtype) + kSampleThreads - 1) / kSampleThreads;
    const int aimed = (kSampleGrid + rows - 1) / rows;
    return std::max(least_slices(vocab, dtype), std::min({most, useful, aimed}));
}
// Slices of all rows that no call of up to `rows` rows goes beyond, whatever its type.
int64_t most_slices(int rows, int vocab, int most) {
    return std::max<int64_t>((int64_t)rows * least_slices(vocab, MOE_F32),
                             std::min<int64_t>((int64_t)rows * most, (int64_t)kSampleGrid + rows));
}
// The same of rows that have several slices: histograms and lists of the others (32 KB each)
// do not leave LDS.
int64_t most_of_several(int rows, int vocab, int most) {
    return most_slices(least_slices(vocab, MOE_F32) > 1 ? rows : std::min(rows, kSampleGrid - 1), vocab,
                       most);
}
struct SampleSpace {
    size_t hist, sums, list, slices, borders, listed, all;
};
// hists, lists: of those slices and draws how many have a histogram and a list there.
SampleSpace sample_space(int64_t slices, int64_t hists, int64_t draws, int64_t lists, int rows) {
    SampleSpace s;
    s.hist = 0;
    s.sums = s.hist + sizeof(uint64_t) * kSampleBins * hists;
    s.list = s.sums + sizeof(double) * kSampleWaves * kSampleSlots * draws;
    s.slices = s.list + sizeof(uint64_t) * kSampleList * lists;
    s.borders = s.slices + sizeof(SampleSlice) * slices;
    s.listed = s.borders + sizeof(SampleBorder) * rows;
    s.all = s.listed + sizeof(int32_t) * draws;
    return s;
}

}  // namespace

extern "C" {

moe_status moe_kv_append_rotated(const moe_kv_cache *kv, int32_t layer, const moe_rotary *rotary,
                                 const void *q, int64_t q_token_stride, int64_t q_head_stride,
                                 int32_t q_heads, const void *k, const void *v, int32_t dtype,
                                 int64_t token_stride, int64_t head_stride, int32_t tokens,
                                 const int32_t *cu, int32_t batch, const int32_t *granted,
                                 void *q_out, moe_stream_t stream) {
    moe_status s = moe_kv_validate(kv);
    if (s != MOE_OK) return s;
    if (!rotary || !rotary->turns || !aligned(rotary->turns, 8) || rotary->first < 0 ||
        rotary->rot < 16 || rotary->first % 16 || rotary->rot % 16 ||
        (rotary->interleaved & ~1) || rotary->first > kv->head_dim ||
        rotary->rot > kv->head_dim - rotary->first)
        return MOE_ERR_INVALID_ARG;
    if (layer < 0 || layer >= kv->layers || q_heads < 1 || tokens < 0 || batch < 0 ||
        batch > kv->seqs || tokens > kMaxRows)
        return MOE_ERR_INVALID_ARG;
    if (q_heads > 1 << 20 || tokens > kMaxGrid256) return MOE_ERR_UNSUPPORTED;   // (a token each)
    if (!cu && tokens != batch) return MOE_ERR_INVALID_ARG;
    if (tokens == 0 || batch == 0) return MOE_OK;
    if (!q || !k || !v || !q_out || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) ||
        !aligned(q_out, 16))
        return MOE_ERR_INVALID_ARG;
    if ((s = check_types(*kv, dtype)) != MOE_OK) return s;
    if ((s = check_strides(q_token_stride, q_head_stride, q_heads, kv->head_dim)) != MOE_OK) return s;
    if ((s = check_strides(token_stride, head_stride, kv->kv_heads, kv->head_dim)) != MOE_OK)
        return s;
    // In place only where every result has its own query's place.
    if (q_out == q && ((tokens > 1 && q_token_stride != (int64_t)q_heads * kv->head_dim) ||
                       (q_heads > 1 && q_head_stride != kv->head_dim)))
        return MOE_ERR_INVALID_ARG;
    int cus;
    if ((s = compute_units(&cus)) != MOE_OK) return s;
    RotaryArgs a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_out = q_out;
    a.kc = plane(*kv, layer, 0);
    a.vc = plane(*kv, layer, 1);
    a.turns = rotary->turns;
    a.tables = kv->tables;
    a.lengths = kv->lengths;
    a.cu = cu;
    a.granted = granted;
    a.k_scale = kv->k_scale;
    a.v_scale = kv->v_scale;
    a.q_token = q_token_stride;
    a.q_head = q_head_stride;
    a.kv_token = token_stride;
    a.kv_head = head_stride;
    a.amplitude = rotary->amplitude;
    a.tokens = tokens;
    a.batch = batch;
    a.pages = kv->pages;
    a.cols = kv->cols;
    a.page_log2 = log2_of(kv->page);
    a.q_heads = q_heads;
    a.kv_heads = kv->kv_heads;
    a.head_dim = kv->head_dim;
    a.first = rotary->first;
    a.rot = rotary->rot;
    // Tokens of few heads share a workgroup and those of many take several, where
    // that still, or only then, fills the chip.
    const int rounds = ((q_heads + 2 * kv->kv_heads) * (kv->head_dim / 16) + kRotaryThreads - 1) /
                       kRotaryThreads;
    a.per_block = std::max(1, std::min({kRotaryTokens, tokens / (8 * cus), (8 + rounds - 1) / rounds}));
    a.parts = tokens < 4 * cus ? std::max(1, std::min(rounds, 4 * cus / tokens)) : 1;
    a.parts = std::min(a.parts, 1 << 15);
    const dim3 grid((tokens + a.per_block - 1) / a.per_block, a.parts);
    return with_types(dtype, kv->dtype == MOE_E4M3, [&](auto t, auto f8) {
        constexpr bool kF8 = decltype(f8)::value;
        if (rotary->interleaved)
            k_kv_rotary<decltype(t), kF8, true><<<grid, kRotaryThreads, 0, stream>>>(a);
        else
            k_kv_rotary<decltype(t), kF8, false><<<grid, kRotaryThreads, 0, stream>>>(a);
        return launched();
    });
}

moe_status moe_sample_workspace(int32_t rows, int32_t vocab, size_t *workspace, size_t *counters) {
    if (rows < 1 || vocab < 1 || !workspace || !counters) return MOE_ERR_INVALID_ARG;
    if (rows > kMaxRows / kSampleMaxDraws || vocab > kMaxVocab) return MOE_ERR_UNSUPPORTED;
    *workspace = sample_space(most_slices(rows, vocab, kSampleMaxSlices),
                              most_of_several(rows, vocab, kSampleMaxSlices),
                              most_slices(rows, vocab, kSampleMaxDraws),
                              most_of_several(rows, vocab, kSampleMaxDraws), rows).all;
    *counters = sizeof(uint32_t) * (size_t)rows;
    return MOE_OK;
}

moe_status moe_sample(const void *x, int32_t dtype, int64_t row_stride, int32_t rows, int32_t vocab,
                      const float *u, const moe_sampling *filters, int32_t *token, float *logprob,
                      void *workspace, uint32_t *counters, moe_stream_t stream) {
    if ((dtype != MOE_BF16 && dtype != MOE_FP16 && dtype != MOE_F32) || rows < 0 || vocab < 1 ||
        !filters || (rows > 1 && row_stride < vocab))
        return MOE_ERR_INVALID_ARG;
    if (rows > kMaxRows / kSampleMaxDraws || vocab > kMaxVocab || row_stride > 1ll << 40)
        return MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MOE_OK;
    if (!x || !u || !token || !logprob || !aligned(x, dtype == MOE_F32 ? 4 : 2) || !aligned(u, 4) ||
        !aligned(token, 4) || !aligned(logprob, 4) || !aligned(filters->temperature, 4) ||
        !aligned(filters->top_p, 4) || !aligned(filters->min_p, 4) || !aligned(filters->top_k, 4))
        return MOE_ERR_INVALID_ARG;
    if (!workspace || !counters || !aligned(workspace, 16) || !aligned(counters, 16))
        return MOE_ERR_WORKSPACE;
    int cus;
    moe_status s = compute_units(&cus);
    if (s != MOE_OK) return s;
    SampleArgs a = {};
    a.slices_n = sample_slices(rows, vocab, dtype, kSampleMaxSlices);
    a.draws = sample_slices(rows, vocab, dtype, kSampleMaxDraws);
    const int64_t slices = (int64_t)a.slices_n * rows, draws = (int64_t)a.draws * rows;
    const SampleSpace space = sample_space(slices, a.slices_n > 1 ? slices : 0, draws,
                                           a.draws > 1 ? draws : 0, rows);
    char *ws = (char *)workspace;
    a.x = x;
    a.u = u;
    a.temperature = filters->temperature;
    a.top_p = filters->top_p;
    a.min_p = filters->min_p;
    a.top_k = filters->top_k;
    a.temperature_all = filters->temperature_all;
    a.top_p_all = filters->top_p_all;
    a.min_p_all = filters->min_p_all;
    a.top_k_all = filters->top_k_all;
    a.token = token;
    a.logprob = logprob;
    a.hist = (uint64_t *)(ws + space.hist);
    a.sums = (double *)(ws + space.sums);
    a.list = (uint64_t *)(ws + space.list);
    a.borders = (SampleBorder *)(ws + space.borders);
    a.slices = (SampleSlice *)(ws + space.slices);
    a.listed = (int32_t *)(ws + space.listed);
    a.counters = counters;
    a.stride = rows > 1 ? row_stride : 0;
    a.rows = rows;
    a.vocab = vocab;
    auto per_wave = [&](int slices) {
        return (row_chunks(vocab, dtype) + slices * kSampleWaves - 1) / (slices * kSampleWaves);
    };
    a.chunks = per_wave(a.slices_n);
    a.draw_chunks = per_wave(a.draws);
    const int grid = rows * a.draws;
    // Filters for all rows are known here; those by row are not.
    const bool plain = !a.top_k && !a.top_p && !a.min_p && !(a.top_k_all > 0 && a.top_k_all < vocab) &&
                       !(a.top_p_all < 1.f) && !(a.min_p_all > 0.f);
    auto go = [&](auto plainly, auto scan, auto draw) {
        if (plain) {
            plainly<<<grid, kSampleThreads, 0, stream>>>(a);
            return launched();
        }
        scan<<<rows * a.slices_n, kSampleThreads, 0, stream>>>(a);
        const moe_status r = launched();
        if (r != MOE_OK) return r;
        draw<<<grid, kSampleThreads, 0, stream>>>(a);
        return launched();
    };
    if (dtype == MOE_F32) return go(k_sample_plain<kSampleF32>, k_sample_scan<kSampleF32>, k_sample_draw<kSampleF32>);
    if (dtype == MOE_FP16) return go(k_sample_plain<1>, k_sample_scan<1>, k_sample_draw<1>);
    return go(k_sample_plain<0>, k_sample_scan<0>, k_sample_draw<0>);
}

}  // extern "C"
