// shared.hip - host side of decode over shared prefixes: the plan, argument checks, and
// their part of the C ABI declared in include/moe_serve.h.
//
// Two launches.  The first has two kinds of workgroups.  Some multiply the queries of all
// members of a group with the keys of their prefix, as prompts do: the rows (member, query
// head) of a kv head are taken 128 at a time, so that prefix keys are read once for 128
// rows instead of once for each member.  The others decode what each sequence has behind
// the prefix.  The second launch joins the partial results of both.
//
// Device time of the two launches, us: 64 sequences, 56 heads on 8, prefix 8192 and tails up
// to 512: 38 and 7; four groups of 16, e4m3, prefixes up to 32768 and tails up to 1000: 83 and
// 8; 32 sequences, 14 heads on 2, prefix 131072 and tails up to 300: 51 and 12.  Prefixes are bound
// as prompts are (vector and matrix instructions), after some 7 us to their first keys;
// tails by memory.  As launches of their own, each on the whole chip, they took 29 + 24,
// 66 + 24 and 49 + 8.
#include "serve_host.h"

#include "attn_decode.h"
#include "attn_prompt.h"
#include "attn_shared.h"

using namespace moe::serve;

namespace {

// The fewest tiles of 64 keys that a workgroup takes, and the most parts of a prefix: every
// part is read again by the join.
constexpr int kSharedTiles = 4, kSharedParts = 128;
// Bytes of keys and values that reading prefixes apart has to spare: it takes some 16 us at
// least, in which a prefix that is read again comes from the caches.  Decode of each
// sequence by itself, and shared, us, 7 heads on each kv head: 7 MB (8 of 2000, 1 kv head)
// 11 and 16; 29 MB (8 of 8192, 1; 8 of 4096, 2; 8 of 1024, 8) 18 and 18, 21 and 16, 13 and 16;
// 34 MB (2 of 32768, 2) 20 and 24; 59 MB (8 of 8192, 2) 24 and 18; 66 MB (64 of 256, 8) 23
// and 17; 126 MB (16 of 4096, 8, e4m3) 28 and 18; 264 MB (64 of 1024, 8) 35 and 18.  Within
// windows, counted as above (members by window, kv heads): 0.3 MB (2 by 64, 8) 11 and 16;
// 32 MB (16 by 512, 8) 13 and 19; 34 MB (64 by 128, 8) 19 and 20; 59 MB (8 by 8192, 2) 24 and
// 21; 66 MB (32 by 2048, 2) 17 and 23; 118 MB (8 by 4096, 8) 21 and 22; 133 MB (64 by 512, 8)
// 27 and 20, behind longer tails, which leave less of the window to the prefix, 28 and 28; 261
// MB (32 by 8192, 2) 34 and 23; 1058 MB (64 by 4096, 8) 85 and 35.  Bytes alone do not decide
// it: a few microseconds are lost on either side of the border (one by one 29 MB of 8
// sequences took 13 to 21, 60 MB 17 to 24, by how many parts their rows were cut into).
constexpr int64_t kSharedLeast = 40000000;
// What the two kinds of work take on the whole chip, us: a first tile of either, 128 rows
// times 64 keys for each dimension, a byte.
constexpr double kStartUs = 7., kPrefixUs = 4.1e-5, kByteUs = 2e-7;

size_t prefix_floats(const moe_attn_shared &p) {
    return (size_t)kPromptRows * (p.head_dim + 2) * p.slots * p.kv_heads;
}
int head_groups(const moe_kv_cache &kv, const moe_attn_config &c) {
    return (c.q_heads / kv.kv_heads + 15) / 16;
}
size_t round16(size_t n) { return (n + 15) / 16 * 16; }

}  // namespace

extern "C" {

moe_status moe_attn_share(const moe_kv_cache *kv, const moe_attn_config *c, int32_t batch,
                          int32_t groups, const int32_t *cu, const int32_t *members,
                          const int32_t *prefix, int64_t least, moe_attn_shared *plan,
                          int32_t *data) {
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
    bool worth = true;
    auto apart = [&](int g) {
        return worth && cu[g + 1] - cu[g] > 1 && prefix[g] > 0 &&
               (c->window == 0 || c->sinks <= prefix[g]);
    };
    // Most positions that a sequence sees of n: a window's, and the sinks.
    auto seen_of = [&](int64_t n) {
        return c->window > 0 ? std::min<int64_t>(n, (int64_t)c->window + c->sinks) : n;
    };
    const double row_bytes = (double)plane_bytes(*kv) / kv->pages / kv->page * 2;
    double spared = 0.0;
    for (int g = 0; g < groups; ++g)
        if (apart(g))
            spared += (double)(cu[g + 1] - cu[g] - 1) *
                      seen_of(std::min<int64_t>(prefix[g], most)) * row_bytes;
    worth = spared >= (double)(least < 0 ? kSharedLeast : least);
    auto tiles_of = [&](int g) { return ((cu[g + 1] - cu[g]) * group + kPromptRows - 1) / kPromptRows; };
    // Tiles of keys that all members together see of a prefix: none begins its window before
    // the shortest one does, which has the whole prefix as a rule, and a window begins
    // within a tile.
    auto tiles_in = [](int64_t n) { return (n + kPromptKeys - 1) / kPromptKeys; };
    auto keys_of = [&](int g) {
        const int64_t all = tiles_in(std::min<int64_t>(prefix[g], most));
        return c->window > 0 ? std::min(all, tiles_in(c->window) + 1 + tiles_in(c->sinks)) : all;
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
    // The workgroups that prefixes get: their share of the time that both kinds of work take,
    // but half at least, since tails may be far shorter than those that are planned for.
    int64_t work = 0, longest = 0, behind = 0;
    for (int g = 0; g < groups; ++g)
        if (apart(g)) {
            work += tiles_of(g) * keys_of(g);
            longest = std::max<int64_t>(longest, prefix[g]);
            behind += cu[g + 1] - cu[g];
        }
    const double tails = (double)behind * seen_of(std::max<int64_t>(0, c->longest - longest)) +
                         (double)(batch - behind) * seen_of(c->longest);
    const double t_prefix = kStartUs + kPrefixUs * work * kv->kv_heads * kv->head_dim;
    const double t_tail = kStartUs + tails * row_bytes * kByteUs;
    const double part = std::max(0.5, t_prefix / (t_prefix + t_tail));
    const int64_t slots =
        std::max<int64_t>(1, (int64_t)(prompt_slots(kv->head_dim) * part) / kv->kv_heads);
    const int64_t aim = units_with(1ll << 40) <= slots ? slots : 4 * slots;
    int64_t lo = kSharedTiles - 1, hi = 1ll << 26;      // (units_with falls)
    if (units_with(kSharedTiles) <= aim) hi = kSharedTiles;
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) / 2;
        if (units_with(mid) <= aim) hi = mid;
        else lo = mid;
    }
    const int64_t share = hi, units = units_with(share);
    int64_t tiles = 0;
    int parts = 0;       // most of a group's
    for (int g = 0; g < groups; ++g)
        if (apart(g)) {
            tiles += tiles_of(g);
            parts = std::max(parts, (int)parts_of(g, share));
        }
    if (units * kv->kv_heads > kMaxGrid256 ||
        tiles * (kv->head_dim / 8) * kv->kv_heads > kMaxGrid256)
        return MOE_ERR_UNSUPPORTED;
    // The longest that is left for each sequence by itself.
    int64_t shortest = total == batch && groups ? most : 0;
    for (int g = 0; g < groups; ++g)
        if (cu[g + 1] > cu[g]) shortest = std::min<int64_t>(shortest, apart(g) ? prefix[g] : 0);
    *plan = {};
    plan->batch = batch;
    plan->q_heads = c->q_heads;
    plan->kv_heads = kv->kv_heads;
    plan->head_dim = kv->head_dim;
    plan->units = (int32_t)(units * kv->kv_heads);
    plan->slots = (int32_t)units;
    plan->members = (int32_t)total;
    plan->window = c->window;
    plan->sinks = c->sinks;
    plan->tiles = (int32_t)tiles;
    plan->parts = parts;
    plan->tail = (int32_t)std::max<int64_t>(1, c->longest - shortest);
    plan->ints = 8 * (plan->units + tiles) + batch + total;
    if (!data) return MOE_OK;
    SharedUnit *unit = (SharedUnit *)data, *tile = unit + plan->units;
    int32_t *prefixes = (int32_t *)(tile + tiles);
    std::fill(prefixes, prefixes + batch, -1);
    int64_t at = 0;
    for (int g = 0; g < groups; ++g) {
        const int n = cu[g + 1] - cu[g];
        for (int i = cu[g]; i < cu[g + 1]; ++i) {
            int32_t &p = prefixes[members[i]];
            if (p >= 0) return MOE_ERR_INVALID_ARG;   // named twice
            p = apart(g) ? prefix[g] : 0;
        }
        if (!apart(g)) continue;
        // All row tiles of a part and head read the same keys: workgroups go round the eight
        // XCDs, so they are eight apart, on one of them.
        const int its = (int)tiles_of(g), parts = (int)parts_of(g, share);
        const int streams = parts * kv->kv_heads;
        auto make = [&](int t, int part, int head) {
            return SharedUnit{cu[g], n, prefix[g], t * kPromptRows, part, parts,
                              (int32_t)at + t * parts + part, head};
        };
        for (int s0 = 0; s0 < streams; s0 += 8)
            for (int t = 0; t < its; ++t)
                for (int y = s0; y < std::min(s0 + 8, streams); ++y)
                    *unit++ = make(t, y / kv->kv_heads, y % kv->kv_heads);
        for (int t = 0; t < its; ++t) *tile++ = make(t, 0, 0);
        at += (int64_t)its * parts;
    }
    for (int b = 0; b < batch; ++b) prefixes[b] = std::max(prefixes[b], 0);
    std::copy(members, members + total, prefixes + batch);
    return MOE_OK;
}

moe_status moe_attn_shared_workspace(const moe_kv_cache *kv, const moe_attn_config *c,
                                     const moe_attn_shared *plan, size_t *workspace,
                                     size_t *counters) {
    const moe_status s = moe_attn_workspace(kv, c, 0, workspace, counters);
    if (s != MOE_OK) return s;
    if (!plan || plan->q_heads != c->q_heads || plan->kv_heads != kv->kv_heads ||
        plan->head_dim != kv->head_dim || plan->slots < 0 || plan->batch < 1 ||
        plan->batch > c->batch || plan->tail > c->longest)
        return MOE_ERR_INVALID_ARG;
    *workspace = round16(*workspace) + sizeof(float) * prefix_floats(*plan) +
                 sizeof(SharedTail) * plan->batch * kv->kv_heads * head_groups(*kv, *c);
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
        plan->window != c->window || plan->sinks != c->sinks || plan->units < 0 ||
        plan->tiles < 0 || plan->slots < 0 ||
        plan->tail > c->longest)    // (more parts than the workspace has room for)
        return MOE_ERR_INVALID_ARG;
    // Nothing is read apart: as any decode.
    if (plan->units == 0)
        return moe_attn_decode(kv, c, layer, q, dtype, token_stride, head_stride, plan->batch, out,
                               lse, workspace, counters, stream);
    size_t decode_bytes, counter_bytes;
    if ((s = moe_attn_workspace(kv, c, 0, &decode_bytes, &counter_bytes)) != MOE_OK) return s;
    if (!workspace || !counters) return MOE_ERR_WORKSPACE;
    AttnArgs a = attn_args(*kv, *c, layer);
    // One unit behind the prefixes for each compute unit: tails are short, and prefixes are in the
    // same launch (one a compute unit, half and twice as many, us: 64 tails of up to 512, 56
    // heads on 8: 39.9, 39.4 and 40.9; 4 groups of 16 up to 1000, e4m3: 85.3, 85.5 and 85.4).
    a.split = std::max(1, std::min(decode_split(*kv, *c, plan->tail),
                                   kPlanCus / (a.kv_heads * a.head_groups)));
    const int64_t grid = ((int64_t)a.split + plan->batch) * a.kv_heads * a.head_groups;
    if (grid + plan->units > kMaxGrid256) return MOE_ERR_UNSUPPORTED;
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
    a.prefix_units = plan->units;
    a.batch = plan->batch;
    a.shared_tails = (SharedTail *)(a.shared_part + prefix_floats(*plan));
    a.shared_units = (const SharedUnit *)plan->data;
    a.shared_tiles = a.shared_units + plan->units;
    a.prefixes = (const int32_t *)(a.shared_tiles + plan->tiles);
    a.members = a.prefixes + plan->batch;
    return with_types(dtype, kv->dtype == MOE_E4M3, [&](auto t, auto f8) {
        return with_dim(kv->head_dim, [&](auto d) {
            typedef decltype(t) T;
            constexpr bool kF8 = decltype(f8)::value;
            constexpr int D = decltype(d)::value;
            k_attn_decode<T, kF8, D, true>
                <<<(int)(plan->units + grid), kDecodeThreads, 0, stream>>>(a);
            const moe_status r = launched();
            if (r != MOE_OK) return r;
            const int64_t join = (int64_t)plan->tiles * 4 * (D / 32) * kv->kv_heads;
            // Up to 32 parts are two rounds of loads; more are taken by four times the waves.
            if (plan->parts <= 32)
                k_attn_join<T, kF8, D, 1><<<(int)join, kJoinThreads, 0, stream>>>(a);
            else
                k_attn_join<T, kF8, D, 4><<<(int)join, 4 * kJoinThreads, 0, stream>>>(a);
            return launched();
        });
    });
}

}  // extern "C"
