// attn_decode.h - attention of one new token per sequence over the paged cache.
//
// For a kv head h the G = q_heads / kv_heads query heads that share it are the
// 16 columns of one MFMA operand (more than 16: several head groups).  Keys
// run in blocks of 32: S^T = K q^T (two 16x16 tiles, keys down, heads across)
// and O^T += V^T P^T.  The first product leaves lane l with the keys 4g..4g+3
// (g = l / 16) of both tiles for head l % 16, which is what the second takes
// as its column operand when its reduction runs over the keys in that order:
// weights never leave their lane.  V is read row by row (16 lanes read the
// whole row of one key, each E = D / 16 elements) and its pairs of keys are
// put together in registers, so MFMA j gives the outputs d = E i + j.  No
// shared memory until the waves meet, once, at the end.
//
// Every lane keeps the running maximum and sum of its head; the maximum is a
// lazy one: accumulators are rescaled only when a score exceeds it by more
// than T::kSlack, which is rare after the first block.  The weights enter the
// second product as a pair hi + lo of 16-bit values: the matrix cores have the
// time (the kernel waits for memory), and the output is then off by its own
// rounding alone.
//
// Work split.  A unit is a run of blocks of one (sequence, kv head).  Lengths
// live on the device, so every workgroup reads them and finds its own unit:
// blocks per unit = all visible blocks / the units aimed at, a multiple of
// the workgroup's waves, and more where one long row would be joined from
// hundreds of parts (one sequence of 100000, 8 heads on 1: 782 parts 101 us, 87
// parts 28 us).  Rows that take one unit are written by it; of the
// units of a longer row the last to arrive joins the others' results.
//
// Bound by memory: 64 sequences of up to 8192 on an e4m3 cache, 570 MB, take 125
// us (4.6 TB/s), two of up to 131072 in bf16, 823 MB, 156 us (5.3 TB/s).  One
// sequence of 1500 takes 9.1 us: a chain of length, pages, keys, the store of a
// part, its arrival and the join, each about a memory latency.  Long single rows
// do not fill the chip (25000 positions, 8 heads on 1: 17 us, 100000: 27, of
// which memory needs 2.5 and 10): one workgroup joins their parts.  No registers
// are spilled but at head_dim 256 on a 16-bit cache (17).
#pragma once

#include "serve_common.h"

namespace moe {
namespace serve {

constexpr int kDecodeWaves = 4;
constexpr int kDecodeThreads = 64 * kDecodeWaves;
constexpr int kDecodeBlock = 32;

// Where element j of lane column i sits in the head: E consecutive ones, except
// 96 e4m3 codes, whose 6 bytes per lane would not be aligned (4 + 2 instead).
template <bool F8, int D>
__device__ __forceinline__ int dim_of(int i, int j) {
    if constexpr (F8 && D == 96) return j < 4 ? 4 * i + j : 64 + 2 * i + j - 4;
    return D / 16 * i + j;
}

template <class T, bool F8, int D>
struct DecodeTile {
    static constexpr int KS = D / 32;                        // MFMA steps of a key row
    static constexpr int E = D / 16;                         // elements of a value row per lane
    static constexpr int KW = F8 ? 2 * KS : 4 * KS;          // dwords of a key row per lane
    static constexpr int VW = F8 ? (E + 3) / 4 : E / 2;      // ... of a value row
    static constexpr int ES = F8 ? 1 : 2;
    uint32_t k[2][KW];
    uint32_t v[8][VW];

    // base: position 16t of the block, of both keys and values.
    __device__ __forceinline__ void load_k(const char *t0, const char *t1, int c, int g) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const char *p = (t ? t1 : t0) + c * (D * ES);
            if constexpr (F8) {
#pragma unroll
                for (int j = 0; j < KS / 2; ++j) load_words<4>(&k[t][4 * j], p + 64 * j + 16 * g);
                if constexpr (KS % 2) load_words<2>(&k[t][2 * KS - 2], p + 32 * (KS - 1) + 8 * g);
            } else {
#pragma unroll
                for (int j = 0; j < KS; ++j) load_words<4>(&k[t][4 * j], p + 64 * j + 16 * g);
            }
        }
    }
    // First element of the eight that MFMA step j takes from lane group g.
    static __device__ __forceinline__ int k_dim(int j, int g) {
        if constexpr (F8) {
            if (KS % 2 && j == KS - 1) return 32 * j + 8 * g;
            return 64 * (j / 2) + 16 * g + 8 * (j & 1);
        }
        return 32 * j + 8 * g;
    }
    __device__ __forceinline__ u32x4 k_op(int t, int j) const {
        if constexpr (F8) {
            const uint32_t a = k[t][2 * j], b = k[t][2 * j + 1];
            return (u32x4){T::template from_e4m3<false>(a), T::template from_e4m3<true>(a),
                           T::template from_e4m3<false>(b), T::template from_e4m3<true>(b)};
        } else {
            return (u32x4){k[t][4 * j], k[t][4 * j + 1], k[t][4 * j + 2], k[t][4 * j + 3]};
        }
    }
    __device__ __forceinline__ void load_v(const char *t0, const char *t1, int c, int g) {
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const char *p = (r < 4 ? t0 : t1) + (4 * g + (r & 3)) * (D * ES);
            if constexpr (F8 && D == 96) {
                v[r][0] = *(const uint32_t *)(p + 4 * c);
                v[r][1] = *(const uint16_t *)(p + 64 + 2 * c);
            } else {
                load_words<VW>(v[r], p + c * (E * ES));
            }
        }
    }
    // Elements 2j and 2j + 1 of key r.
    template <int J>
    __device__ __forceinline__ uint32_t v_pair(int r) const {
        if constexpr (F8)
            return T::template from_e4m3<(J & 1) != 0>(v[r][J / 2]);
        else
            return v[r][J];
    }
};

template <class T, bool F8, int D, int J>
__device__ __forceinline__ void pv(const DecodeTile<T, F8, D> &t, u32x4 p_hi, u32x4 p_lo,
                                   f32x4 *o) {
    if constexpr (J < D / 32) {
        uint32_t w[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) w[r] = t.template v_pair<J>(r);
        u32x4 a, b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], 0x05040100u);
            b[i] = __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], 0x07060302u);
        }
        o[2 * J] = T::mfma16(a, p_hi, o[2 * J]);
        o[2 * J + 1] = T::mfma16(b, p_hi, o[2 * J + 1]);
        o[2 * J] = T::mfma16(a, p_lo, o[2 * J]);
        o[2 * J + 1] = T::mfma16(b, p_lo, o[2 * J + 1]);
        pv<T, F8, D, J + 1>(t, p_hi, p_lo, o);
    }
}

// The sums over keys among whose values some are not finite, from 2 J on.
// each(f) calls f(t0, t1, sees) for every block: its two halves of 16 values and
// a bit for each of this lane's eight keys; put(j, r, sum) takes them.
template <class T, int D, int J, class Each, class Put>
__device__ __forceinline__ void sum_not_finite(Each each, Put put) {
    if constexpr (J < D / 32) {
        const int c = lane_id() & 15, g = lane_id() >> 4;
        constexpr uint32_t one2 = T::kOne | T::kOne << 16;
        const u32x4 ones = {one2, one2, one2, one2};
        f32x4 x[2][2] = {{zero4(), zero4()}, {zero4(), zero4()}};
        each([&](const char *t0, const char *t1, uint32_t sees) {
            uint32_t w[8];
#pragma unroll
            for (int r = 0; r < 8; ++r)
                w[r] = sees >> r & 1 ? *(const uint32_t *)((r < 4 ? t0 : t1) +
                                                           (4 * g + (r & 3)) * (2 * D) +
                                                           c * (D / 8) + 4 * J)
                                     : 0u;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                u32x4 a, b;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t m0 = marks_of<T>(w[2 * i], s), m1 = marks_of<T>(w[2 * i + 1], s);
                    a[i] = __builtin_amdgcn_perm(m1, m0, 0x05040100u);
                    b[i] = __builtin_amdgcn_perm(m1, m0, 0x07060302u);
                }
                x[s][0] = T::mfma16(a, ones, x[s][0]);
                x[s][1] = T::mfma16(b, ones, x[s][1]);
            }
        });
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool pos = x[0][j][r] != 0.f, neg = x[1][j][r] != 0.f;
                if (pos || neg) put(2 * J + j, r, sum_of_marks(pos, neg));
            }
        sum_not_finite<T, D, J + 1>(each, put);
    }
}

struct DecodeUnit {
    int b, n;        // sequence (-1: none), its length as far as its table goes
    int first;       // of its window's positions (0: no window)
    Visible vis;
    int i0, i1;      // visible blocks of this unit
    int unit0, parts;  // the row's first unit (per kv head), and how many there are
};

// The unit of index `want` among all sequences' units (per kv head).
__device__ __forceinline__ DecodeUnit find_unit(const AttnArgs &a, int want) {
    const int lane = lane_id();
    const int most = a.cols << a.page_log2;
    // The token's position is the length's, also where the table is too short for it.
    auto first_of = [&](int n) { return a.window > 0 ? max(0, n - a.window) : 0; };
    auto vis_of = [&](int n) { return visible<5>(min(n, most), first_of(n), a.sinks); };
    int sum = 0, longest = 0, n0 = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
        const int b = b0 + lane;
        n0 = b < a.batch ? max(a.lengths[b], 0) : 0;
        const int total = vis_of(n0).total;
        sum += total;
        longest = max(longest, total);
    }
    sum = (int)uniform(wave_sum_i(sum));
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) longest = max(longest, __shfl_xor(longest, m));
    int c = (sum + a.split - 1) / a.split;
    c = max(1, (c + kDecodeWaves - 1) / kDecodeWaves) * kDecodeWaves;
    // Joining a part takes 0.1 us, in one workgroup; a round of a unit's waves
    // over four blocks takes half of one: no more parts than balance the two.
    const int least = (int)uniform((uint32_t)__builtin_amdgcn_sqrtf(0.45f * (float)longest));
    c = max(c, least / kDecodeWaves * kDecodeWaves);
    DecodeUnit u;
    u.b = -1;
    int base = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
        const int b = b0 + lane;
        const int n = a.batch <= 64 ? n0 : b < a.batch ? max(a.lengths[b], 0) : 0;
        const Visible vis = vis_of(n);
        const int parts = b < a.batch ? max(1, (vis.total + c - 1) / c) : 0;
        int all;
        const int at = base + wave_excl_scan(parts, &all);
        const uint64_t mine = __ballot(want >= at && want < at + parts);
        if (mine) {
            const int l = __builtin_ctzll(mine);
            u.b = b0 + l;
            const int length = __builtin_amdgcn_readlane(n, l);
            u.n = min(length, most);
            u.first = first_of(length);
            u.unit0 = __builtin_amdgcn_readlane(at, l);
            u.parts = __builtin_amdgcn_readlane(parts, l);
            u.vis = vis_of(length);
            u.i0 = (want - u.unit0) * c;
            u.i1 = min(u.vis.total, u.i0 + c);
            break;
        }
        base += (int)uniform(all);
    }
    return u;
}

template <class T, bool F8, int D>
__global__ __launch_bounds__(kDecodeThreads, 2) void k_attn_decode(const AttnArgs a) {
    typedef DecodeTile<T, F8, D> Tile;
    constexpr int W = kDecodeWaves, KS = Tile::KS, E = Tile::E, ES = Tile::ES;
    constexpr int kRow = D + 4;
    __shared__ __attribute__((aligned(16))) float s_o[W][16][kRow];
    __shared__ float s_m[W][16], s_l[W][16], s_den[16];
    __shared__ uint32_t s_last;

    const int lane = lane_id(), wave = wave_index(), c = lane & 15, g = lane >> 4;
    const int heads = a.kv_heads * a.head_groups;
    const int hh = (int)blockIdx.x % heads, su = (int)blockIdx.x / heads;
    const DecodeUnit u = find_unit(a, su);
    if (u.b < 0) return;
    const int h = hh / a.head_groups, hg = hh % a.head_groups;
    const int head0 = h * a.group + 16 * hg;             // first query head of the columns
    const int n_heads = min(16, a.group - 16 * hg);

    // Query columns: head c, the elements each key operand multiplies.
    u32x4 q[KS];
    {
        const uint16_t *qp = (const uint16_t *)a.q + u.b * a.q_token +
                             (head0 + (c < n_heads ? c : 0)) * a.q_head;
#pragma unroll
        for (int j = 0; j < KS; ++j) {
            q[j] = ld16(qp + Tile::k_dim(j, g));
            if (c >= n_heads) q[j] = (u32x4){0, 0, 0, 0};
        }
    }
    const float c2 = a.scale * (F8 && a.k_scale ? a.k_scale[h] : 1.f);

    f32x4 o[E];
#pragma unroll
    for (int j = 0; j < E; ++j) o[j] = zero4();
    float m = kNoMax, l = 0.f;

    const int32_t *row = a.tables + (int64_t)u.b * a.cols;
    const int64_t head_bytes = (int64_t)D * ES << a.page_log2;   // of one head of one page
    const int in_page = (1 << a.page_log2) - 1;
    const int first = u.first;
    struct Ids {
        int key;
        uint32_t p[2];
    };
    auto ids_of = [&](int i) {
        Ids x;
        x.key = 32 * visible_block(u.vis, i);
        x.p[0] = (uint32_t)row[x.key >> a.page_log2];
        x.p[1] = (uint32_t)row[min((x.key + 16) >> a.page_log2, a.cols - 1)];
        return x;
    };
    auto at = [&](const void *base, const Ids &x, int t) {
        const uint32_t p = x.p[t] < (uint32_t)a.pages ? x.p[t] : 0u;
        return (const char *)base + ((int64_t)p * a.kv_heads + h) * head_bytes +
               ((x.key + 16 * t) & in_page) * (D * ES);
    };

    // Whether key 16 (r / 4) + 4 g + r % 4 of a block is seen.
    auto sees_of = [&](const Ids &x, int r) {
        const int key = x.key + 16 * (r >> 2) + 4 * g + (r & 3);
        return (key < u.n) & (x.p[r >> 2] < (uint32_t)a.pages) & ((key >= first) | (key < a.sinks));
    };

    int i = u.i0 + wave;
    if (i < u.i1) {
        Tile t;
        Ids now = ids_of(i), next = ids_of(min(i + W, u.i1 - 1));
        t.load_k(at(a.k, now, 0), at(a.k, now, 1), c, g);
        t.load_v(at(a.v, now, 0), at(a.v, now, 1), c, g);
        for (;;) {
            const bool more = i + W < u.i1;
            const Ids after = ids_of(min(i + 2 * W, u.i1 - 1));
            f32x4 s[2] = {zero4(), zero4()};
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                s[0] = T::mfma16(t.k_op(0, j), q[j], s[0]);
                s[1] = T::mfma16(t.k_op(1, j), q[j], s[1]);
            }
            if (more) t.load_k(at(a.k, next, 0), at(a.k, next, 1), c, g);

            float x[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) x[r] = s[r >> 2][r & 3] * c2;
            // A block that is not seen as a whole: hidden keys get no weight,
            // and their values, which may be anything, are taken as zero.
            const bool whole = now.key + 32 <= u.n && now.p[0] < (uint32_t)a.pages &&
                               now.p[1] < (uint32_t)a.pages &&
                               (now.key >= first || now.key + 32 <= a.sinks);
            if (!whole) {
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const bool sees = sees_of(now, r);
                    x[r] = sees ? x[r] : -__builtin_inff();
#pragma unroll
                    for (int w = 0; w < Tile::VW; ++w) t.v[r][w] = sees ? t.v[r][w] : 0u;
                }
            }
            float top = x[0];
#pragma unroll
            for (int r = 1; r < 8; ++r) top = fmaxf(top, x[r]);
            if (__any(top > m + T::kSlack)) {
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                const float to = fmaxf(m, top), f = exp2_(m - to);
                m = to;
                l *= f;
#pragma unroll
                for (int j = 0; j < E; ++j) o[j] *= f;
            }
            u32x4 hi, lo;
#pragma unroll
            for (int r = 0; r < 8; r += 2) {
                // The rounded scores less their rounded maximum: a fused product
                // would leave the maximum's own rounding, which is no small number
                // where scores are large.
#pragma clang fp contract(off)
                const float p0 = exp2_(x[r] - m + T::kOff), p1 = exp2_(x[r + 1] - m + T::kOff);
                l += p0 + p1;
                hi[r / 2] = T::pack(p0, p1);
                lo[r / 2] = T::pack(p0 - T::lo(hi[r / 2]), p1 - T::hi(hi[r / 2]));
            }
            pv<T, F8, D, 0>(t, hi, lo, o);
            if (!more) break;
            t.load_v(at(a.v, next, 0), at(a.v, next, 1), c, g);
            i += W;
            now = next;
            next = after;
        }
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
    }

    // The waves meet.
    if (c < n_heads) {
        if (g == 0) {
            s_m[wave][c] = m;
            s_l[wave][c] = l;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int j = 0; j < E; ++j) s_o[wave][c][dim_of<F8, D>(4 * g + r, j)] = o[j][r];
    }
    // A visible value that is infinite has made NaN of its sums: the second half of
    // a pair of weights is zero or negative, and weights and factors may be too
    // small for their type.  By the definition they are positive, so the sum is
    // that infinity, or NaN where both are seen.  Rare, so values are read again,
    // without haste.  (e4m3 has no infinities, and NaN stays.)
    if constexpr (!F8) {
        float zero = 0.f;   // or NaN
#pragma unroll
        for (int j = 0; j < E; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) zero = fmaf(o[j][r], 0.f, zero);
        if (__any(zero != zero))
            sum_not_finite<T, D, 0>(
                [&](auto take) {
#pragma unroll 1
                    for (int y = u.i0 + wave; y < u.i1; y += W) {
                        const Ids x = ids_of(y);
                        uint32_t sees = 0;
#pragma unroll
                        for (int r = 0; r < 8; ++r) sees |= (uint32_t)sees_of(x, r) << r;
                        take(at(a.v, x, 0), at(a.v, x, 1), sees);
                    }
                },
                [&](int j, int r, float x) {
                    if (c < n_heads) s_o[wave][c][dim_of<F8, D>(4 * g + r, j)] = x;
                });
    }
    __syncthreads();
    const float v_scale = F8 && a.v_scale ? a.v_scale[h] : 1.f;
    const int64_t out_row = (int64_t)u.b * a.kv_heads * a.group + head0;
    auto write = [&](int head, int d, f32x4 x) {
        uint32_t *op = (uint32_t *)a.out + ((out_row + head) * D + d) / 2;
        const u32x2 w = {T::pack(x[0] * v_scale, x[1] * v_scale),
                         T::pack(x[2] * v_scale, x[3] * v_scale)};
        *(u32x2 *)op = w;
    };
    auto write_lse = [&](int head, float x) { a.lse[out_row + head] = x; };
    constexpr int64_t kSlot = 16 * (D + 2);
    float *mine = a.part + ((int64_t)su * heads + hh) * kSlot;
    for (int x = threadIdx.x; x < n_heads * (D / 4); x += kDecodeThreads) {
        const int head = x / (D / 4), d = 4 * (x % (D / 4));
        float top = s_m[0][head];
#pragma unroll
        for (int w = 1; w < W; ++w) top = fmaxf(top, s_m[w][head]);
        f32x4 sum = zero4();
        float den = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float f = part_factor(s_m[w][head] - top);
            sum += ldf4(&s_o[w][head][d]) * f;
            den += s_l[w][head] * f;
        }
        if (u.parts == 1) {
            write(head, d, den != 0.f ? sum * (1.f / den) : zero4());
            if (d == 0)
                write_lse(head, den != 0.f ? (top + log2_(den) - T::kOff) * kLn2
                                           : -__builtin_inff());
        } else {
            buf_st16<true>(buf_rsrc(mine), 4u * (head * D + d), __builtin_bit_cast(u32x4, sum));
            if (d == 0) {
                store_agent(mine + 16 * D + head, top);
                store_agent(mine + 16 * D + 16 + head, den);
            }
        }
    }
    if (u.parts == 1) return;

    // Arrival: this unit's stores are complete before it is counted.
    wait_vm_all();
    __syncthreads();
    uint32_t *counter = a.counters + (int64_t)u.b * heads + hh;
    if (threadIdx.x == 0)
        s_last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (s_last != (uint32_t)u.parts - 1) return;
    if (threadIdx.x == 0) store_agent(counter, 0u);
    join_parts<T, D, kDecodeThreads>(a.part + ((int64_t)u.unit0 * heads + hh) * kSlot,
                                     kSlot * heads, u.parts, n_heads, 16, s_m[0], s_den, write,
                                     write_lse);
}

}  // namespace serve
}  // namespace moe
