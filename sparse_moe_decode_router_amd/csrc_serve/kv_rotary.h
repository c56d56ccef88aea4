// kv_rotary.h - new keys and values into their pages, the keys and the queries
// beside them turned by their positions on the way.
//
// A pair (x0, x1) of frequency f at position p becomes a (x0 cos pf - x1 sin pf),
// a (x1 cos pf + x0 sin pf).  Positions reach 2^31, where a product p f in 32 bits
// would be off by whole turns: it is formed in 64 bits, in turns (f / 2 pi comes
// from the caller), and only what is left of it below an eighth of a turn goes on
// in 32, into the power series of sine and cosine.  That is done once per token
// and pair, by the workgroup, and kept in LDS for all heads.
//
// An item is two chunks of eight elements of one head: in a part that is turned
// chunks i and i + r / 16, which hold whole pairs in both orders (neighbours, or
// halves r / 2 apart), elsewhere two chunks as far apart.  Lanes next to each other
// take chunks next to each other.  An item reads both of its chunks before it
// writes them, so queries may be turned in place.
//
// Memory bounds it: 20750 tokens, 56 heads on 8 of 128, bf16, are 765 MB read and
// written in 154 us, 4.98 TB/s, where a copy reaches 5.07.  A workgroup has up to eight
// tokens there, so that finding a sequence and the cosines are waited for once in eight.
// Where tokens are few a token is cut into parts, since the chain of loads (length,
// page, row) and not the bytes is what takes the time: 64 tokens of 56 heads on 8
// into e4m3 pages 4.6 us, one of 7 heads on 1 2.9.
#pragma once

#include "serve_common.h"

namespace moe {
namespace serve {

struct RotaryArgs {
    const void *q, *k, *v;
    void *q_out, *kc, *vc;         // kc, vc: the layer's pages
    const double *turns;           // [rot / 2]
    const int32_t *tables, *lengths, *cu;
    const int32_t *granted;        // or NULL: positions that a sequence was given
    const float *k_scale, *v_scale;
    int64_t q_token, q_head, kv_token, kv_head;   // strides in elements
    float amplitude;
    int32_t tokens, batch, pages, cols, page_log2, q_heads, kv_heads, head_dim;
    int32_t first, rot;
    int32_t per_block;             // tokens of a workgroup; 1 where `parts` > 1
    int32_t parts;                 // workgroups of a token
};

constexpr int kRotaryThreads = 256;
constexpr int kRotaryTokens = 8;   // most tokens of a workgroup
constexpr int kRotaryMaxDim = 256;

// cos and sin of `turns` turns.
__device__ __forceinline__ void cos_sin(double turns, float *c, float *s) {
    const double quarter = __builtin_rint(4.0 * turns);
    const float x = 6.2831853071795865f * (float)(turns - 0.25 * quarter);   // up to pi / 4
    const int k = (int)(quarter - 4.0 * __builtin_floor(0.25 * quarter));    // 0 .. 3
    const float y = x * x;
    // Power series: what is left out is below 2^-28 of the sine and 2^-24.7 of the cosine
    // (x^10 / 10! at pi / 4), as much as a rounding.
    const float sn = x + x * y * (-1.f / 6 + y * (1.f / 120 + y * (-1.f / 5040 + y * (1.f / 362880))));
    const float cs = 1.f + y * (-0.5f + y * (1.f / 24 + y * (-1.f / 720 + y * (1.f / 40320))));
    const float a = k & 1 ? sn : cs, b = k & 1 ? cs : sn;
    *c = k == 1 || k == 2 ? -a : a;
    *s = k & 2 ? -b : b;
}

template <class T, bool F8, bool Pairs>
__global__ __launch_bounds__(kRotaryThreads) void k_kv_rotary(const RotaryArgs a) {
    __shared__ __attribute__((aligned(16))) float s_cos[kRotaryTokens][kRotaryMaxDim / 2];
    __shared__ __attribute__((aligned(16))) float s_sin[kRotaryTokens][kRotaryMaxDim / 2];
    __shared__ int64_t s_at[kRotaryTokens];   // row of the first head's page, or -1
    __shared__ int s_pos[kRotaryTokens];      // -1: none, -2: a row of no sequence
    const int t0 = (int)blockIdx.x * a.per_block, n_tok = min(a.per_block, a.tokens - t0);
    const int half = a.rot >> 1;
    if ((int)threadIdx.x < n_tok) {
        const int t = t0 + (int)threadIdx.x;
        int b = t, pos, n_new = 1;
        bool ours = true;
        if (a.cu) {
            int lo = 0, hi = a.batch;   // the last b with cu[b] <= t
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (a.cu[mid] <= t) lo = mid;
                else hi = mid;
            }
            b = lo;
            const int from = a.cu[b], to = a.cu[b + 1];
            ours = t >= from && t < to;
            n_new = to - from;
            pos = (int)max((int64_t)a.lengths[b] - ((int64_t)to - t), (int64_t)-1);
        } else {
            pos = max(a.lengths[b], 0) - 1;
        }
        int64_t at = -1;
        if (ours && pos >= 0 && pos < a.cols << a.page_log2 &&
            !(a.granted && a.granted[b] < n_new)) {
            const uint32_t page = (uint32_t)a.tables[(int64_t)b * a.cols + (pos >> a.page_log2)];
            if (page < (uint32_t)a.pages)
                at = (((int64_t)page * a.kv_heads) << a.page_log2) + (pos & ((1 << a.page_log2) - 1));
        }
        s_at[threadIdx.x] = at;
        s_pos[threadIdx.x] = ours ? pos : -2;
    }
    __syncthreads();
    for (int x = threadIdx.x; x < n_tok * half; x += kRotaryThreads) {
        const int i = x / half, j = x - i * half;
        float c, s;
        cos_sin((double)s_pos[i] * a.turns[j], &c, &s);
        s_cos[i][j] = c * a.amplitude;
        s_sin[i][j] = s * a.amplitude;
    }
    __syncthreads();

    const int per_head = a.head_dim >> 4, turned = a.rot >> 4;
    const int kv_from = a.q_heads * per_head, v_from = kv_from + a.kv_heads * per_head;
    const int per_token = v_from + a.kv_heads * per_head;
    const int plain = (a.head_dim - a.rot) >> 4;    // items of a head that are not turned
    const int step = kRotaryThreads * a.parts;
    int i = 0, x = (int)threadIdx.x + kRotaryThreads * (int)blockIdx.y;
    for (;;) {
        while (x >= per_token) {
            x -= per_token;
            if (++i >= n_tok) return;
        }
        const int pos = s_pos[i];
        const int64_t at = s_at[i], t = t0 + i;
        const int item = x;
        x += step;
        const bool is_q = item < kv_from, is_v = item >= v_from;
        if (is_q ? pos == -2 : at < 0) continue;
        const int y = item - (is_q ? 0 : is_v ? v_from : kv_from);
        const int h = y / per_head, u = y - h * per_head;
        const bool turn = !is_v && u < turned;
        // The item's two chunks.
        int d0, d1;
        if (is_v) {
            d0 = 8 * u;
            d1 = d0 + 8 * per_head;
        } else if (turn) {
            d0 = a.first + 8 * u;
            d1 = d0 + half;
        } else {
            d0 = 8 * (u - turned);
            d1 = d0 + 8 * plain;
            d0 += d0 >= a.first ? a.rot : 0;
            d1 += d1 >= a.first ? a.rot : 0;
        }
        const uint16_t *from = is_q ? (const uint16_t *)a.q + t * a.q_token + h * a.q_head
                                    : (const uint16_t *)(is_v ? a.v : a.k) + t * a.kv_token +
                                          h * a.kv_head;
        u32x4 w[2] = {ld16(from + d0), ld16(from + d1)};
        f32x4 f[2][2];
        // A row without a position (a slot that no sequence holds) stays as it is.
        const bool now = turn && pos >= 0;
        if (now) {
            float v[2][8];
#pragma unroll
            for (int z = 0; z < 2; ++z)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[z][2 * e] = T::lo(w[z][e]);
                    v[z][2 * e + 1] = T::hi(w[z][e]);
                }
            // Pairs of the first chunk from 4 u on, of the second half / 2 further; or
            // both chunks' pairs from 8 u on.
            const int j0 = Pairs ? 4 * u : 8 * u, j1 = Pairs ? j0 + (half >> 1) : j0 + 4;
            const f32x4 c0 = ldf4(&s_cos[i][j0]), s0 = ldf4(&s_sin[i][j0]);
            const f32x4 c1 = ldf4(&s_cos[i][j1]), s1 = ldf4(&s_sin[i][j1]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float c = e < 4 ? c0[e] : c1[e - 4], s = e < 4 ? s0[e] : s1[e - 4];
                float &p = Pairs ? v[e >> 2][2 * (e & 3)] : v[0][e];
                float &r = Pairs ? v[e >> 2][2 * (e & 3) + 1] : v[1][e];
                const float p0 = p, r0 = r;
                p = p0 * c - r0 * s;
                r = r0 * c + p0 * s;
            }
#pragma unroll
            for (int z = 0; z < 2; ++z)
#pragma unroll
                for (int e = 0; e < 8; ++e) f[z][e >> 2][e & 3] = v[z][e];
        }
        if (F8 && !is_q) {
            const float *scales = is_v ? a.v_scale : a.k_scale;
            const float scale = scales ? scales[h] : 1.f;
            uint8_t *to = (uint8_t *)(is_v ? a.vc : a.kc) +
                          (at + ((int64_t)h << a.page_log2)) * a.head_dim;
#pragma unroll
            for (int z = 0; z < 2; ++z)
                *(u32x2 *)(to + (z ? d1 : d0)) =
                    now ? (u32x2){to_e4m3(f[z][0], scale), to_e4m3(f[z][1], scale)}
                        : to_e4m3<T>(w[z], scale);
            continue;
        }
        if (now) {
#pragma unroll
            for (int z = 0; z < 2; ++z)
                w[z] = (u32x4){T::pack(f[z][0][0], f[z][0][1]), T::pack(f[z][0][2], f[z][0][3]),
                               T::pack(f[z][1][0], f[z][1][1]), T::pack(f[z][1][2], f[z][1][3])};
        }
        uint16_t *to = is_q ? (uint16_t *)a.q_out + (t * a.q_heads + h) * a.head_dim
                            : (uint16_t *)(is_v ? a.vc : a.kc) +
                                  (at + ((int64_t)h << a.page_log2)) * a.head_dim;
        *(u32x4 *)(to + d0) = w[0];
        *(u32x4 *)(to + d1) = w[1];
    }
}

}  // namespace serve
}  // namespace moe
