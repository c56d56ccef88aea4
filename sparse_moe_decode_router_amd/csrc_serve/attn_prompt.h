// attn_prompt.h - attention of the new tokens of several sequences (prompts, or
// chunks of them) over the paged cache, causal, with an optional window and
// first positions that stay visible.
//
// For a kv head the rows of all its G query heads are packed, token by token
// (row = token * G + head): a tile of 128 rows spans 128 / G tokens, so that
// under a window it reads little more than the window itself.  A workgroup
// takes one row tile; its four waves own 32 rows each, as the columns of
// 32x32x16 MFMAs, and share tiles of 64 keys and values in LDS: S^T = K q^T,
// O^T += V^T P^T.  As in decode, the weights are where the second product
// wants them without leaving their lane; V^T is read from the row-major tile
// with transposing LDS reads.
//
// Tiles are double-buffered.  16-bit caches are copied straight into LDS (no
// registers), 16-byte chunk q of row r at position q ^ swizzle(r), which makes
// both the row reads of K (16 rows, one chunk) and the transposed reads of V
// (4 rows, 4 chunks) hit every bank once; e4m3 caches are converted on the way
// through registers.  Only tiles at the edge of what some row sees are masked.
//
// Few rows and many keys: the tiles of a row group are split over several
// workgroups, the last of which joins their results (as in decode).
#pragma once

#include "serve_common.h"

namespace moe {
namespace serve {

constexpr int kPromptThreads = 256;
constexpr int kPromptRows = 128;
constexpr int kPromptKeys = 64;

template <int D>
struct PromptTile {
    static constexpr int kRowBytes = D <= 64 ? 128 : D <= 128 ? 256 : 512;
    static constexpr int kSlots = kRowBytes / 16;   // 16-byte positions of a row
    static constexpr int kChunks = D / 8;           // 16-byte chunks it holds
    static constexpr int kBytes = kPromptKeys * kRowBytes;
    static __device__ __forceinline__ int swizzle(int r) {
        if constexpr (D == 64) return 4 * ((r >> 1) & 1) + ((r >> 2) & 3);
        return 4 * (r & 3) + ((r >> 2) & 3);
    }
    static __device__ __forceinline__ int byte_of(int r, int chunk) {
        return r * kRowBytes + 16 * (chunk ^ swizzle(r));
    }
};

// The number of row tiles of a sequence with `tokens` new tokens.
__device__ __forceinline__ int row_tiles(int tokens, int group) {
    return (int)(((int64_t)tokens * group + kPromptRows - 1) / kPromptRows);
}

typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ u32x2 read_transposed(const char *p) {
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p));
}

// 64 lanes bring 16 bytes each from base + off (off per lane) straight into
// LDS: lane l's to lds + 16 l.  In assembly and without any output: behind the
// builtin the compiler waits for the copy before the next read of LDS, also of
// another buffer.  Whoever reads the copy waits for vmcnt itself.
__device__ __forceinline__ void copy_to_lds(const void *base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(off), "s"(base)
                 : "memory", "m0");
}
__device__ __forceinline__ uint32_t lds_address(const char *p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char *)p;
}

// What is not finite in two values: 1 (sign 0) or 2 (sign 1) marks, as values
// that are one where v is +inf (or -inf) or NaN and zero elsewhere.
template <class T>
__device__ __forceinline__ uint32_t marks_of(uint32_t v, uint32_t sign) {
    uint32_t out = 0;
#pragma unroll
    for (int z = 0; z < 32; z += 16) {
        const uint32_t h = v >> z & 0xFFFFu;
        out |= (T::odd(h) && (T::nan(h) || h >> 15 == sign) ? T::kOne : 0u) << z;
    }
    return out;
}
template <class T>
__device__ __forceinline__ uint32_t finite_of(uint32_t v) {
    return (T::odd(v) ? 0u : v & 0xFFFFu) | (T::odd(v >> 16) ? 0u : v & 0xFFFF0000u);
}

template <class T, bool F8, int D>
__global__ __launch_bounds__(kPromptThreads, D <= 128 ? 2 : 1) void k_attn_prompt(
    const AttnArgs a) {
    typedef PromptTile<D> Tile;
    constexpr int KS = D / 16, DT = D / 32;
    __shared__ __attribute__((aligned(1024))) char s_k[2][Tile::kBytes];
    __shared__ __attribute__((aligned(1024))) char s_v[2][Tile::kBytes];
    __shared__ float s_m[kPromptRows], s_den[kPromptRows];
    __shared__ uint32_t s_last;
    __shared__ int s_odd;

    const int tid = threadIdx.x, lane = lane_id(), wave = wave_index();
    const int col = lane & 31, half = lane >> 5;

    // The row tile: blockIdx = (tile * kv_heads + h) * split + part.
    const int part = (int)blockIdx.x % a.split;
    const int h = (int)blockIdx.x / a.split % a.kv_heads;
    const int want = (int)blockIdx.x / a.split / a.kv_heads;
    int b = -1, tile = 0, tiles = 0, tok0 = 0, n_new = 0, n = 0;
    {
        int base = 0;
        for (int b0 = 0; b0 < a.batch; b0 += 64) {
            const int bb = b0 + lane;
            int from = 0, to = 0;
            if (bb < a.batch) {
                from = min(max(a.cu[bb], 0), a.tokens);
                to = min(max(a.cu[bb + 1], from), a.tokens);
            }
            const int mine = row_tiles(to - from, a.group);
            int all;
            const int at = base + wave_excl_scan(mine, &all);
            const uint64_t found = __ballot(want >= at && want < at + mine);
            if (found) {
                const int l = __builtin_ctzll(found);
                b = b0 + l;
                tiles = __builtin_amdgcn_readlane(mine, l);
                tile = want - __builtin_amdgcn_readlane(at, l);
                tok0 = __builtin_amdgcn_readlane(from, l);
                n_new = __builtin_amdgcn_readlane(to, l) - tok0;
                break;
            }
            base += (int)uniform(all);
        }
    }
    if (b < 0) return;
    // The length as the caller counts it: a table that is too short hides
    // positions (n_seen), it does not move the new tokens.
    n = max((int)uniform(a.lengths[b]), 0);
    const int n_seen = min(n, a.cols << a.page_log2);
    const int row0 = (tiles - 1 - tile) * kPromptRows;  // late rows, which see most, first
    const int rows = min(kPromptRows, n_new * a.group - row0);
    const int past = n - n_new;
    const int pos_lo = past + row0 / a.group, pos_hi = past + (row0 + rows - 1) / a.group;

    // This lane's row.
    const int my = row0 + min(32 * wave + col, rows - 1);
    const int my_tok = my / a.group, pos = past + my_tok;
    const int from = a.window > 0 ? pos - a.window : -1;        // sees keys above it
    const int64_t out_row =
        (int64_t)(tok0 + my_tok) * a.kv_heads * a.group + h * a.group + (my - my_tok * a.group);
    u32x4 q[KS];
    {
        const uint16_t *qp = (const uint16_t *)a.q + (tok0 + my_tok) * a.q_token +
                             (h * a.group + (my - my_tok * a.group)) * a.q_head + 8 * half;
#pragma unroll
        for (int j = 0; j < KS; ++j) q[j] = ld16(qp + 16 * j);
    }
    // A scale of the cache may be anything: zero stands for the smallest factor
    // (so that a hidden score stays infinite), and a negative one turns the
    // order of the scores round.
    float c2 = a.scale * (F8 && a.k_scale ? a.k_scale[h] : 1.f);
    if (F8 && c2 == 0.f) c2 = 1e-37f;
    const float hidden = F8 && c2 < 0.f ? __builtin_inff() : -__builtin_inff();

    // Tiles of keys that some row of this tile sees.
    const int end = max(0, min(n_seen, pos_hi + 1));
    const Visible vis =
        visible<6>(end, a.window > 0 ? max(0, pos_lo - a.window + 1) : 0, a.sinks);
    const int chunk = max(1, (vis.total + a.split - 1) / a.split);
    const int parts = max(1, (vis.total + chunk - 1) / chunk);
    if (part >= parts) return;
    const int i0 = part * chunk, i1 = min(vis.total, i0 + chunk);

    const int32_t *table = a.tables + (int64_t)b * a.cols;
    constexpr int ES = F8 ? 1 : 2;
    const int64_t head_bytes = (int64_t)D * ES << a.page_log2;
    const int in_page = (1 << a.page_log2) - 1;
    // The pages of a tile's four groups of 16 keys, by scalar loads (the tables
    // are not written here): they wait for nothing of the vector memory.  Wave w
    // brings the keys of group w.
    typedef __attribute__((address_space(4))) const int32_t const_i32;
    const_i32 *table_c = (const_i32 *)(uintptr_t)table;
    struct Pages {
        uint32_t p[4];
    };
    auto pages_of = [&](int i) {
        const int key = (int)uniform(64 * visible_block(vis, i));
        Pages x;
#pragma unroll
        for (int y = 0; y < 4; ++y)
            x.p[y] = (uint32_t)table_c[min((key + 16 * y) >> a.page_log2, a.cols - 1)];
        return x;
    };
    auto row_of = [&](const void *base, const Pages &x, int i) {
        const int key = (int)uniform(64 * visible_block(vis, i) + 16 * wave);
        const uint32_t w = wave;
        uint32_t p = w == 0 ? x.p[0] : w == 1 ? x.p[1] : w == 2 ? x.p[2] : x.p[3];
        p = p < (uint32_t)a.pages ? p : 0u;
        return (const char *)base + ((int64_t)p * a.kv_heads + h) * head_bytes +
               (key & in_page) * (D * ES);
    };
    // Rows x RPI .. of a wave's share, and the piece a lane brings of them.
    constexpr int RPI = 64 / Tile::kSlots, CP = 16 / RPI;
    uint32_t copy_off[F8 ? 1 : CP];
    if constexpr (!F8) {
#pragma unroll
        for (int x = 0; x < CP; ++x) {
            const int r = RPI * x + lane / Tile::kSlots;
            const int ch = (lane % Tile::kSlots) ^ Tile::swizzle(r);
            copy_off[x] = ch < Tile::kChunks ? r * (2 * D) + 16 * ch : ~0u;
        }
    }
    auto copy_in = [&](const void *base, const char *dst, const Pages &pg, int i) {
        const char *src = row_of(base, pg, i);
        const uint32_t to = uniform(lds_address(dst) + 16 * wave * Tile::kRowBytes);
#pragma unroll
        for (int x = 0; x < CP; ++x) {
            if (Tile::kSlots == Tile::kChunks || copy_off[x] != ~0u)
                copy_to_lds(src, copy_off[x], to + RPI * x * Tile::kRowBytes);
        }
    };
    // e4m3: a lane's share of 16 rows is 16 D / 64 codes, in chunks of 8.
    constexpr int NC = F8 ? D / 32 : 1;
    u32x2 raw_k[NC], raw_v[NC];
    auto fetch = [&](const void *base, u32x2 *raw, const Pages &pg, int i) {
        const char *src = row_of(base, pg, i);
#pragma unroll
        for (int x = 0; x < NC; ++x) raw[x] = *(const u32x2 *)(src + 8 * (64 * x + lane));
    };
    auto convert = [&](const u32x2 *raw, char *dst) {
#pragma unroll
        for (int x = 0; x < NC; ++x) {
            const int r = (64 * x + lane) / Tile::kChunks, ch = (64 * x + lane) % Tile::kChunks;
            *(u32x4 *)(dst + Tile::byte_of(16 * wave + r, ch)) =
                (u32x4){T::template from_e4m3<false>(raw[x][0]), T::template from_e4m3<true>(raw[x][0]),
                        T::template from_e4m3<false>(raw[x][1]), T::template from_e4m3<true>(raw[x][1])};
        }
    };

    f32x16 o[DT];
#pragma unroll
    for (int j = 0; j < DT; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[j][r] = 0.f;
    float m = kNoMax, l = 0.f;

    // Where this lane reads, in bytes of a tile.  Chunks of one row differ in
    // address bits of their own (the swizzle depends on the low bits of the row
    // alone), so operand j of K sits at (at_k ^ 32 j), and rows 32 further on at
    // a constant distance.  V is read transposed: a lane group of 16 brings keys
    // k0 .. k0 + 3 (k0 = 16 t + 4 half) of 16 columns, then the same 8 keys on.
    const int key_v = 4 * half + ((lane & 15) >> 2), dim_v = 16 * (lane >> 4 & 1) + 4 * (lane & 3);
    const uint32_t at_k = Tile::byte_of(col, half);
    const uint32_t at_v = Tile::byte_of(key_v, dim_v >> 3) + 2 * (dim_v & 7);
    auto v_op = [&](const char *tile, uint32_t at, int t, int dt) {
        const char *v = tile + 16 * t * Tile::kRowBytes;
        const u32x2 x = read_transposed(v + (at ^ 64 * dt));
        const u32x2 y = read_transposed(v + (at ^ (64 * dt ^ 32)) + 8 * Tile::kRowBytes);
        return (u32x4){x[0], x[1], y[0], y[1]};
    };

    // What rows see of a tile: which groups of 16 keys have a page, and whether
    // every row sees all of it.
    struct Seen {
        int key0;
        uint32_t have;
        bool whole;
    };
    auto seen_of = [&](const Pages &pg, int i) {
        Seen x;
        x.key0 = (int)uniform(64 * visible_block(vis, i));
        x.have = 0;
#pragma unroll
        for (int y = 0; y < 4; ++y) x.have |= pg.p[y] < (uint32_t)a.pages ? 1u << y : 0u;
        x.whole = x.have == 15u && x.key0 + 63 <= pos_lo && x.key0 + 64 <= n_seen &&
                  (a.window <= 0 || x.key0 > pos_hi - a.window || x.key0 + 64 <= a.sinks);
        return x;
    };
    // Scores: keys down (2 x 32), rows across.  Operands are read four at a
    // time, one round ahead of the products that take them.
    auto scores = [&](const char *sk, f32x16 *s) {
        // Opaque, so that the operands' addresses are formed where they are
        // used: kept from tile to tile they take some forty registers.
        uint32_t ak = at_k;
        asm("" : "+v"(ak));
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[u][r] = 0.f;
        u32x4 kb[2][4];
        auto read_k = [&](u32x4 *d, int f0) {
#pragma unroll
            for (int f = 0; f < 4; ++f)
                d[f] = ld16(sk + 32 * ((f0 + f) & 1) * Tile::kRowBytes + (ak ^ 32 * ((f0 + f) >> 1)));
        };
        read_k(kb[0], 0);
#pragma unroll
        for (int f = 0; f < 2 * KS; f += 4) {
            if (f + 4 < 2 * KS) read_k(kb[f / 4 + 1 & 1], f + 4);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int x = 0; x < 4; ++x)
                s[x & 1] = T::mfma32(kb[f / 4 & 1][x], q[(f + x) >> 1], s[x & 1]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto hide = [&](const Seen &see, f32x16 *s) {
        int key0 = see.key0 + 4 * half;  // opaque, as above
        asm("" : "+v"(key0));
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int key = key0 + 32 * u + 8 * (r >> 2) + (r & 3);
                const bool sees = (key <= pos) & (key < n_seen) &
                                  ((key > from) | (key < a.sinks)) &
                                  ((see.have >> (2 * u + (r >> 3)) & 1) != 0);
                s[u][r] = sees ? s[u][r] : hidden;
            }
    };

    if (tid == 0) s_odd = 0;
    Pages now = {}, next = {};
    if (i0 < i1) {
        const Pages p = now = pages_of(i0);
        if constexpr (F8) {
            fetch(a.k, raw_k, p, i0);
            fetch(a.v, raw_v, p, i0);
            convert(raw_k, s_k[0]);
            convert(raw_v, s_v[0]);
        } else {
            copy_in(a.k, s_k[0], p, i0);
            copy_in(a.v, s_v[0], p, i0);
        }
        next = pages_of(min(i0 + 1, i1 - 1));
    }
    for (int i = i0; i < i1; ++i) {
        const int buf = (i - i0) & 1;
        char *sk = s_k[buf], *sv = s_v[buf];
        wait_vm_all();
        __syncthreads();  // this tile is here, and the other buffer is free
        const bool more = i + 1 < i1;
        if (more) {
            if constexpr (F8) {
                fetch(a.k, raw_k, next, i + 1);
                fetch(a.v, raw_v, next, i + 1);
            } else {
                copy_in(a.k, s_k[buf ^ 1], next, i + 1);
                copy_in(a.v, s_v[buf ^ 1], next, i + 1);
            }
        }
        const Seen see = seen_of(now, i);
        now = next;
        next = pages_of(min(i + 2, i1 - 1));
        if (!see.whole) {
            // Values that no row sees become zero, and so do those that are not
            // finite: a row that does not see them would get NaN from them.
            // What they mean for the rows that do see them comes at the end.
            int x0 = tid;  // opaque, as in scores()
            asm("" : "+v"(x0));
#pragma unroll 1
            for (int x = x0; x < kPromptKeys * Tile::kChunks; x += kPromptThreads) {
                const int r = x / Tile::kChunks;
                u32x4 *p = (u32x4 *)(sv + Tile::byte_of(r, x % Tile::kChunks));
                u32x4 w = {0, 0, 0, 0};
                if (see.key0 + r < n_seen && (see.have >> (r >> 4) & 1)) {
                    const u32x4 v = *p;
#pragma unroll
                    for (int y = 0; y < 4; ++y) w[y] = finite_of<T>(v[y]);
                    if (w[0] != v[0] || w[1] != v[1] || w[2] != v[2] || w[3] != v[3]) s_odd = 1;
                }
                *p = w;
            }
            __syncthreads();
        }
        f32x16 s[2];
        scores(sk, s);
        uint32_t av = at_v;
        asm("" : "+v"(av));
        u32x4 vb[2][DT];
        auto read_v = [&](u32x4 *d, int t) {
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) d[dt] = v_op(sv, av, t, dt);
        };
        read_v(vb[0], 0);
        if (!see.whole) hide(see, s);
        float top = s[0][0];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, s[u][r]);
        top *= c2;
        if (F8 && c2 < 0.f) {
            top = -__builtin_inff();
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int r = 0; r < 16; ++r) top = fmaxf(top, s[u][r] * c2);
        }
        if (__any(top > m + T::kSlack)) {
            top = fmaxf(top, __shfl_xor(top, 32));
            const float to = fmaxf(m, top), f = exp2_(m - to);
            m = to;
            l *= f;
#pragma unroll
            for (int j = 0; j < DT; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[j][r] *= f;
        }
        u32x4 p[4];
        const float shift = T::kOff - m;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < 16; r += 2) {
                const float p0 = exp2_(fmaf(s[u][r], c2, shift));
                const float p1 = exp2_(fmaf(s[u][r + 1], c2, shift));
                l += p0 + p1;
                p[2 * u + (r >> 3)][(r & 7) >> 1] = T::pack(p0, p1);
            }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (t < 3) read_v(vb[t + 1 & 1], t + 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) o[dt] = T::mfma32(vb[t & 1][dt], p[t], o[dt]);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (F8) {
            if (more) {
                convert(raw_k, s_k[buf ^ 1]);
                convert(raw_v, s_v[buf ^ 1]);
            }
        }
    }
    __syncthreads();
    if (s_odd) {
        // Values that are not finite, in tiles that some rows see and others do
        // not: a row gets the infinity (for NaN both) of every one on which it
        // has weight.  Rare, so each tile is brought again, without haste.
#pragma unroll 1
        for (int i = i0; i < i1; ++i) {
            const Pages pg = pages_of(i);
            const Seen see = seen_of(pg, i);
            if (see.whole) continue;
            __syncthreads();
            if constexpr (F8) {
                fetch(a.k, raw_k, pg, i);
                fetch(a.v, raw_v, pg, i);
                convert(raw_k, s_k[0]);
                convert(raw_v, s_v[0]);
            } else {
                copy_in(a.k, s_k[0], pg, i);
                copy_in(a.v, s_v[0], pg, i);
            }
            wait_vm_all();
            __syncthreads();
            f32x16 s[2];
            scores(s_k[0], s);
            hide(see, s);
            u32x4 p[4];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int r = 0; r < 16; r += 2)
                    p[2 * u + (r >> 3)][(r & 7) >> 1] =
                        T::pack(exp2_(fmaf(s[u][r], c2, T::kOff - m)),
                                exp2_(fmaf(s[u][r + 1], c2, T::kOff - m)));
#pragma unroll 1
            for (uint32_t sign = 0; sign < 2; ++sign) {
                const float add = sign ? -__builtin_inff() : __builtin_inff();
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) {
                    f32x16 x;
#pragma unroll
                    for (int r = 0; r < 16; ++r) x[r] = 0.f;
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        u32x4 v = v_op(s_v[0], at_v, t, dt);
#pragma unroll
                        for (int y = 0; y < 4; ++y) v[y] = marks_of<T>(v[y], sign);
                        x = T::mfma32(v, p[t], x);
                    }
#pragma unroll
                    for (int r = 0; r < 16; ++r) o[dt][r] += x[r] != 0.f ? add : 0.f;
                }
            }
        }
    }
    l += __shfl_xor(l, 32);

    const bool real = 32 * wave + col < rows;
    if (parts == 1) {
        if (!real) return;
        const float f = l != 0.f ? (F8 && a.v_scale ? a.v_scale[h] : 1.f) / l : 0.f;
        uint16_t *op = (uint16_t *)a.out + out_row * D;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                u32x2 w;
                if (l != 0.f)
                    w = (u32x2){T::pack(o[dt][r] * f, o[dt][r + 1] * f),
                                T::pack(o[dt][r + 2] * f, o[dt][r + 3] * f)};
                else
                    w = (u32x2){0, 0};
                *(u32x2 *)(op + 32 * dt + 2 * r + 4 * half) = w;
            }
        if (half == 0)
            a.lse[out_row] = l != 0.f ? (m + log2_(l) - T::kOff) * kLn2 : -__builtin_inff();
        return;
    }

    constexpr int64_t kSlot = kPromptRows * (D + 2);
    const int64_t group = (int64_t)want * a.kv_heads + h;
    float *slot = a.part + (group * a.split + part) * kSlot;
    if (real) {
        const int r0 = 32 * wave + col;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
            for (int r = 0; r < 16; r += 4)
                buf_st16<true>(buf_rsrc(slot), 4u * (r0 * D + 32 * dt + 2 * r + 4 * half),
                               __builtin_bit_cast(u32x4, (f32x4){o[dt][r], o[dt][r + 1],
                                                                 o[dt][r + 2], o[dt][r + 3]}));
        if (half == 0) {
            store_agent(slot + kPromptRows * D + r0, m);
            store_agent(slot + kPromptRows * D + kPromptRows + r0, l);
        }
    }
    wait_vm_all();
    __syncthreads();
    if (tid == 0)
        s_last = __hip_atomic_fetch_add(a.counters + group, 1u, __ATOMIC_RELAXED,
                                        __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (s_last != (uint32_t)parts - 1) return;
    if (tid == 0) store_agent(a.counters + group, 0u);
    const float v_scale = F8 && a.v_scale ? a.v_scale[h] : 1.f;
    auto out_of = [&](int r) {
        const int at = row0 + r, tok = at / a.group;
        return (int64_t)(tok0 + tok) * a.kv_heads * a.group + h * a.group + (at - tok * a.group);
    };
    join_parts<T, D, kPromptThreads>(
        a.part + group * a.split * kSlot, kSlot, parts, rows, kPromptRows, s_m, s_den,
        [&](int r, int d, f32x4 x) {
            *(u32x2 *)((uint16_t *)a.out + out_of(r) * D + d) =
                (u32x2){T::pack(x[0] * v_scale, x[1] * v_scale),
                        T::pack(x[2] * v_scale, x[3] * v_scale)};
        },
        [&](int r, float x) { a.lse[out_of(r)] = x; });
}

}  // namespace serve
}  // namespace moe
