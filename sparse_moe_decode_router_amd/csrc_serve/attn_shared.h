// attn_shared.h - joins the partial results of attention over shared prefixes: the
// prefix's parts, of groups of sequences, and each sequence's own parts behind it.
//
// Parts of a prefix are as the lanes of k_attn_prompt held them: per 32 rows and 32
// dimensions four blocks of 64 times 16 bytes (row % 32 + 32 (d / 4 % 2)).  A workgroup takes
// 32 rows and 32 dimensions, a wave one of the blocks of a Q-th of the parts: every load of
// a part is a whole block, and sixteen parts of each share are on their way at once.  A
// sequence's own parts are row by row (attn_decode.h).
//
// Loads of what other XCDs wrote bound it: 448 rows of 8 heads 7 us, four groups of 112
// rows of 8 heads 8, 224 rows of 2 heads in 64 parts or so each 12.  In the decode launch,
// by the last arrival of a row, a wave joined its own rows one part after another, and a
// long prefix's 128 parts took 40 us.
#pragma once

#include "serve_common.h"

namespace moe {
namespace serve {

constexpr int kJoinThreads = 256;   // for each of the Q shares

template <class T, bool F8, int D, int Q>
__global__ __launch_bounds__(kJoinThreads * Q) void k_attn_join(const AttnArgs a) {
    constexpr int DT = D / 32;
    constexpr int64_t kOwnSlot = 16 * (D + 2), kSlot = 128 * (D + 2);
    __shared__ f32x4 s_sum[Q][256];
    __shared__ float s_m[Q][256], s_l[Q][256];
    const int lane = lane_id(), col = lane & 31, half = lane >> 5;
    const int block = wave_index() & 3, share = wave_index() >> 2, own_at = threadIdx.x & 255;
    const int h = (int)blockIdx.x % a.kv_heads, rest = (int)blockIdx.x / a.kv_heads;
    const int dt = rest % DT, w = rest / DT % 4;
    const SharedUnit su = a.shared_tiles[rest / (4 * DT)];
    const int rows = su.n_members * a.group, row = su.row0 + 32 * w + col;
    if (su.row0 + 32 * w >= rows) return;
    const int at = min(row, rows - 1), member = at / a.group, g = at - member * a.group;
    const int seq = a.members[su.members + member];
    const int heads = a.kv_heads * a.head_groups, hh = h * a.head_groups + (g >> 4);
    const SharedTail tail = a.shared_tails[(int64_t)seq * heads + hh];
    const int d = 32 * dt + 8 * block + 4 * half;
    const float *own = a.part + ((int64_t)tail.unit0 * heads + hh) * kOwnSlot;
    const float *pre = a.shared_part + ((int64_t)su.slot * a.kv_heads + h) * kSlot + w * 32 * (D + 2);
    const int64_t own_step = kOwnSlot * heads, pre_step = kSlot * a.kv_heads;
    const int ml = 32 * D + col, piece = 256 * (4 * dt + block) + 4 * lane;

    float m = kNoMax, l = 0.f;
    f32x4 sum = zero4();
    // A running maximum over batches of parts.  (A part that is empty for a row may have
    // left no sums at all.)
    auto take = [&](float pm, float pl, f32x4 x, bool is) {
        if (!is || pl == 0.f) return;
        const float f = part_factor(pm - m);
        l = fmaf(pl, f, l);
        sum += x * f;
    };
    auto raise = [&](float to) {
        const float f = part_factor(m - to);
        m = to;
        l *= f;
        sum *= f;
    };
    const int first = su.parts * share / Q;
    const int end = su.parts * (share + 1) / Q;
    for (int u = first; u < end; u += 16) {
        float pm[16], pl[16];
        f32x4 x[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float *p = pre + min(u + j, end - 1) * pre_step;
            pm[j] = p[ml];
            pl[j] = p[ml + 32];
            x[j] = ldf4(p + piece);
        }
        float top = m;
#pragma unroll
        for (int j = 0; j < 16; ++j) top = fmaxf(top, pl[j] != 0.f ? pm[j] : kNoMax);
        if (u > first) raise(top);
        m = top;
#pragma unroll
        for (int j = 0; j < 16; ++j) take(pm[j], pl[j], x[j], u + j < end);
    }
    const int r = g & 15;
    for (int u = share; u < tail.parts; u += Q) {
        const float *p = own + u * own_step;
        const float pm = p[16 * D + r], pl = p[16 * D + 16 + r];
        const f32x4 x = ldf4(p + r * D + d);
        raise(fmaxf(m, pl != 0.f ? pm : kNoMax));
        take(pm, pl, x, true);
    }
    s_sum[share][own_at] = sum;
    s_m[share][own_at] = m;
    s_l[share][own_at] = l;
    __syncthreads();
    if (share || row >= rows) return;
#pragma unroll
    for (int y = 1; y < Q; ++y) {
        const float pl = s_l[y][own_at], pm = s_m[y][own_at];
        raise(fmaxf(m, pl != 0.f ? pm : kNoMax));
        take(pm, pl, s_sum[y][own_at], true);
    }
    const int64_t out_row = ((int64_t)seq * a.kv_heads + h) * a.group + g;
    const float f = l != 0.f ? (F8 && a.v_scale ? a.v_scale[h] : 1.f) / l : 0.f;
    u32x2 o = {0, 0};
    if (l != 0.f)
        o = (u32x2){T::pack(sum[0] * f, sum[1] * f), T::pack(sum[2] * f, sum[3] * f)};
    *(u32x2 *)((uint16_t *)a.out + out_row * D + d) = o;
    if (dt == 0 && block == 0 && half == 0)
        a.lse[out_row] = l != 0.f ? (m + log2_(l) - T::kOff) * kLn2 : -__builtin_inff();
}

}  // namespace serve
}  // namespace moe
