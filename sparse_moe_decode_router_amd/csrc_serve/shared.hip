// shared.hip - host side of decode over shared prefixes: the plan, argument checks, and
// their part of the C ABI declared in include/moe_serve.h.
//
// Two launches.  The first multiplies the queries of all members of a group with the
// keys of their prefix, as prompts do: the rows (member, query head) of a kv head are
// taken 128 at a time, and the prefix in as many parts as fill the chip once.  The
// second is decode over what each sequence has behind the prefix, and joins its
// partial results with the first one's.  Prefix keys are read once for 128 rows instead
// of once for each member.
#include "serve_host.h"

#include "attn_decode.h"
#include "attn_prompt.h"

using namespace moe::serve;

namespace {

// The fewest tiles of 64 keys that a workgroup takes, and the most parts of a prefix: every
// part is read again by the join.
constexpr int kSharedTiles = 4, kSharedParts = 64;

size_t prefix_floats(const moe_attn_shared &p) {
    return (size_t)kPromptRows * (p.head_dim + 2) * p.slots * p.kv_heads;
}
size_t round16(size_t n) { return (n + 15) / 16 * 16; }

}  // namespace

extern "C" {

moe_status moe_attn_share(const moe_kv_cache *kv, const moe_attn_config *c, int32_t batch,
                          int32_t groups, const int32_t *cu, const int32_t *members,
                          const int32_t *prefix, moe_attn_shared *plan, int32_t *data) {
    const moe_status s = moe_attn_validate(kv, c);
    if (s != MOE_OK) return s;
    if (!plan || batch < 1 || batch > c->batch || groups < 0 || groups > batch ||
        (groups && (!cu || !prefix)))
        return MOE_ERR_INVALID_ARG;
    const int64_t group = c->q_heads / kv->kv_heads, most = (int64_t)kv->cols * kv->page;
    int64_t total = 0;
    for (int g = 0; g < groups; ++g) {
        const int64_t n = (int64_t)cu[g + 1] - cu[g];
        if (cu[0] != 0 || n < 0 || prefix[g] < 0 || cu[g + 1] > batch) return MOE_ERR_INVALID_ARG;
        total = cu[g + 1];
        if (n * group > 1ll << 30) return MOE_ERR_UNSUPPORTED;
    }
    if (total && !members) return MOE_ERR_INVALID_ARG;
    for (int i = 0; i < total; ++i)
        if (members[i] < 0 || members[i] >= batch) return MOE_ERR_INVALID_ARG;
    // A prefix that is read apart: one that several share, and that holds all sinks (those
    // behind it would be seen beside a window that is behind them).
    auto apart = [&](int g) {
        return cu[g + 1] - cu[g] > 1 && prefix[g] > 0 && (c->window == 0 || c->sinks <= prefix[g]);
    };
    auto tiles_of = [&](int g) { return ((cu[g + 1] - cu[g]) * group + kPromptRows - 1) / kPromptRows; };
    auto keys_of = [&](int g) {
        return (std::min<int64_t>(prefix[g], most) + kPromptKeys - 1) / kPromptKeys;
    };
    // The smallest share of tiles of keys with which all workgroups fit at once; if none
    // does, four rounds of them.
    auto parts_of = [&](int g, int64_t share) {
        return std::max<int64_t>(1, std::min<int64_t>(kSharedParts, (keys_of(g) + share - 1) / share));
    };
    auto units_with = [&](int64_t share) {
        int64_t n = 0;
        for (int g = 0; g < groups; ++g)
            if (apart(g)) n += tiles_of(g) * parts_of(g, share);
        return n;
    };
    const int64_t slots = std::max(1, prompt_slots(kv->head_dim) / kv->kv_heads);
    const int64_t aim = units_with(1ll << 40) <= slots ? slots : 4 * slots;
    int64_t lo = kSharedTiles - 1, hi = 1ll << 26;      // (units_with falls)
    if (units_with(kSharedTiles) <= aim) hi = kSharedTiles;
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) / 2;
        if (units_with(mid) <= aim) hi = mid;
        else lo = mid;
    }
    const int64_t share = hi, units = units_with(share);
    if (units * kv->kv_heads > kMaxGrid256) return MOE_ERR_UNSUPPORTED;
    // The longest that is left for each sequence by itself.
    int64_t least = total == batch && groups ? most : 0;
    for (int g = 0; g < groups; ++g)
        if (cu[g + 1] > cu[g]) least = std::min<int64_t>(least, apart(g) ? prefix[g] : 0);
    *plan = {};
    plan->batch = batch;
    plan->q_heads = c->q_heads;
    plan->kv_heads = kv->kv_heads;
    plan->head_dim = kv->head_dim;
    plan->units = (int32_t)units;
    plan->slots = (int32_t)units;
    plan->members = (int32_t)total;
    plan->window = c->window;
    plan->sinks = c->sinks;
    plan->tail = (int32_t)std::max<int64_t>(1, c->longest - least);
    plan->ints = 8 * units + 4 * (int64_t)batch + total;
    if (!data) return MOE_OK;
    SharedUnit *unit = (SharedUnit *)data;
    SharedRow *rows = (SharedRow *)(data + 8 * units);
    for (int b = 0; b < batch; ++b) rows[b] = {0, 0, 0, -1};
    int64_t at = 0;
    for (int g = 0; g < groups; ++g) {
        const int n = cu[g + 1] - cu[g];
        const bool is = apart(g);
        const int parts = (int)parts_of(g, share);
        for (int i = 0; i < n; ++i) {
            SharedRow &r = rows[members[cu[g] + i]];
            if (r.member >= 0) return MOE_ERR_INVALID_ARG;   // named twice
            r = is ? SharedRow{prefix[g], (int32_t)at, parts, i} : SharedRow{0, 0, 0, i};
        }
        if (!is) continue;
        // All row tiles of a part are neighbours: they read the same keys.
        const int tiles = (int)tiles_of(g);
        for (int part = 0; part < parts; ++part)
            for (int t = 0; t < tiles; ++t)
                unit[at + part * tiles + t] = {cu[g], n, prefix[g], t * kPromptRows, part, parts,
                                               (int32_t)at + t * parts + part, 0};
        at += (int64_t)tiles * parts;
    }
    for (int b = 0; b < batch; ++b) rows[b].member = std::max(rows[b].member, 0);
    std::copy(members, members + total, data + 8 * units + 4 * (int64_t)batch);
    return MOE_OK;
}

moe_status moe_attn_shared_workspace(const moe_kv_cache *kv, const moe_attn_config *c,
                                     const moe_attn_shared *plan, size_t *workspace,
                                     size_t *counters) {
    const moe_status s = moe_attn_workspace(kv, c, 0, workspace, counters);
    if (s != MOE_OK) return s;
    if (!plan || plan->q_heads != c->q_heads || plan->kv_heads != kv->kv_heads ||
        plan->head_dim != kv->head_dim || plan->slots < 0)
        return MOE_ERR_INVALID_ARG;
    *workspace = round16(*workspace) + sizeof(float) * prefix_floats(*plan);
    return MOE_OK;
}

moe_status moe_attn_decode_shared(const moe_kv_cache *kv, const moe_attn_config *c,
                                  const moe_attn_shared *plan, int32_t layer, const void *q,
                                  int32_t dtype, int64_t token_stride, int64_t head_stride,
                                  void *out, float *lse, void *workspace, uint32_t *counters,
                                  moe_stream_t stream) {
    if (!plan) return MOE_ERR_INVALID_ARG;
    moe_status s = check_attn(kv, c, layer, q, dtype, token_stride, head_stride, plan->batch, out, lse,
                              workspace, counters);
    if (s != MOE_OK) return s;
    if (!plan->data || !aligned(plan->data, 16) || plan->q_heads != c->q_heads ||
        plan->kv_heads != kv->kv_heads || plan->head_dim != kv->head_dim ||
        plan->window != c->window || plan->sinks != c->sinks || plan->units < 0)
        return MOE_ERR_INVALID_ARG;
    size_t decode_bytes, counter_bytes;
    if ((s = moe_attn_workspace(kv, c, 0, &decode_bytes, &counter_bytes)) != MOE_OK) return s;
    if (!workspace || !counters) return MOE_ERR_WORKSPACE;
    AttnArgs a = attn_args(*kv, *c, layer);
    a.split = decode_split(*kv, *c, plan->tail);
    const int64_t grid = ((int64_t)a.split + plan->batch) * a.kv_heads * a.head_groups;
    const int64_t first = (int64_t)plan->units * kv->kv_heads;
    if (grid > kMaxGrid256 || first > kMaxGrid256) return MOE_ERR_UNSUPPORTED;
    int cus;
    if ((s = compute_units(&cus)) != MOE_OK) return s;
    a.q = q;
    a.q_token = token_stride;
    a.q_head = head_stride;
    a.out = out;
    a.lse = lse;
    a.part = (float *)workspace;
    a.shared_part = (float *)((char *)workspace + round16(decode_bytes));
    a.counters = counters;
    a.batch = plan->batch;
    a.shared_units = (const SharedUnit *)plan->data;
    a.shared_rows = (const SharedRow *)(plan->data + 8 * (int64_t)plan->units);
    a.members = plan->data + 8 * (int64_t)plan->units + 4 * (int64_t)plan->batch;
    return with_types(dtype, kv->dtype == MOE_E4M3, [&](auto t, auto f8) {
        return with_dim(kv->head_dim, [&](auto d) {
            typedef decltype(t) T;
            constexpr bool kF8 = decltype(f8)::value;
            constexpr int D = decltype(d)::value;
            if (first) {
                k_attn_prompt<T, kF8, D, true><<<(int)first, kPromptThreads, 0, stream>>>(a);
                const moe_status r = launched();
                if (r != MOE_OK) return r;
            }
            k_attn_decode<T, kF8, D, true><<<(int)grid, kDecodeThreads, 0, stream>>>(a);
            return launched();
        });
    });
}

}  // extern "C"
