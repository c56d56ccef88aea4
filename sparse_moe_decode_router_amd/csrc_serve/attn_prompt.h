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
// Work split.  Few row tiles and many keys: each row tile is split over several
// workgroups.  More row tiles than the chip holds at once: every workgroup
// takes an equal share of all tiles of keys laid end to end, in which a row
// tile counts kPromptFixed more than it has (head_dim 256, 2 x 2000 tokens: 95
// us against 119 with a workgroup per row tile).  Of the parts of a split row
// tile the last to arrive joins the others' results.
//
// What bounds it: the issue of vector and matrix instructions, one after the
// other in each wave, and the clock.  8192 tokens, window 4096, 14 heads take
// 390000 cycles, 204 to 220 us by card (890 to 825 TFLOP/s): matrix cores and
// vector unit are busy 45% of them each, with no bank conflicts to speak of and
// 85% of the reads met in L2.  On an e4m3 cache it is 493000 cycles, 240 us: codes
// are converted on their way into LDS.  Scores of the next tile interleaved with
// this one's exponentials, in one wave, measured no faster (229 against 220
// us, at the time); raising the priority of waves in the second product did (241
// to 220).
//
// Registers: none are spilled on 16-bit caches (one at head_dim 256 in fp16); on
// e4m3 caches 14 at head_dim 128, 13 at 192 and 57 at 256.
#pragma once

#include "serve_common.h"

namespace moe {
namespace serve {

constexpr int kPromptThreads = 256;
constexpr int kPromptRows = 128;
constexpr int kPromptKeys = 64;
// Equal shares: what a row tile costs beside its tiles of keys, in such tiles, and
// the smallest share.
constexpr int kPromptFixed = 6, kPromptLeast = 16;
// A weight is one fused product, 2^(s c - max): exact but for the rounding of the
// maximum, 2^-14 of the weight where that is up to this.  Beyond, s c is rounded
// as the maximum was.
constexpr float kLargeMax = 1024.f;

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

// Reads at an address of LDS.
__device__ __forceinline__ u32x2 read_transposed(uint32_t at) {
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)at));
}
__device__ __forceinline__ u32x4 read_lds16(uint32_t at) {
    return *(const __attribute__((address_space(3))) u32x4 *)at;
}

// 64 lanes bring N times 16 bytes each straight into LDS: lane l's x-th from base +
// off[x] (+ 1024 x with Stride) to lds + 1024 x + 16 l.  In assembly and without any
// output: behind the builtin the compiler waits for the copy before the next
// read of LDS, also of another buffer.  Whoever reads the copy waits for vmcnt
// itself.  The compiler does not look into it for hazards either: a base that a
// vector instruction has just put into scalar registers (a restored spill) may
// be read five wait states later.
template <int N>
__device__ __forceinline__ void copy_to_lds(const void *base, const uint32_t *off, uint32_t lds) {
    if constexpr (N == 1)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2"
                     :
                     : "s"(lds), "v"(off[0]), "s"(base)
                     : "memory", "m0");
    if constexpr (N == 2)
        asm volatile(
            "s_mov_b32 m0, %0\n\ts_nop 4\n\t"
            "global_load_lds_dwordx4 %1, %3\n\t"
            "global_load_lds_dwordx4 %2, %3 offset:1024"
            :
            : "s"(lds), "v"(off[0]), "v"(off[1]), "s"(base)
            : "memory", "m0");
    if constexpr (N == 4)
        asm volatile(
            "s_mov_b32 m0, %0\n\ts_nop 4\n\t"
            "global_load_lds_dwordx4 %1, %5\n\t"
            "global_load_lds_dwordx4 %2, %5 offset:1024\n\t"
            "global_load_lds_dwordx4 %3, %5 offset:2048\n\t"
            "global_load_lds_dwordx4 %4, %5 offset:3072"
            :
            : "s"(lds), "v"(off[0]), "v"(off[1]), "v"(off[2]), "v"(off[3]), "s"(base)
            : "memory", "m0");
}
__device__ __forceinline__ uint32_t lds_address(const char *p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char *)p;
}

// Two values, those that are not finite as zero.
template <class T>
__device__ __forceinline__ uint32_t finite_of(uint32_t v) {
    return (T::odd(v) ? 0u : v & 0xFFFFu) | (T::odd(v >> 16) ? 0u : v & 0xFFFF0000u);
}

// The kernel's arguments, read again by what follows: kept in scalar registers from
// the start on, they have to make room for others in lanes of vector registers.
typedef __attribute__((address_space(4))) const AttnArgs PromptArgs;
__device__ __forceinline__ PromptArgs &prompt_args() {
    PromptArgs *a = (PromptArgs *)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(a));
    return *a;
}

template <class T, bool F8, int D>
__global__ __launch_bounds__(kPromptThreads, D <= 128 ? 2 : 1) void k_attn_prompt(
    const AttnArgs) {
    typedef PromptTile<D> Tile;
    constexpr int KS = D / 16, DT = D / 32;
    __shared__ __attribute__((aligned(1024))) char s_k[2][Tile::kBytes];
    __shared__ __attribute__((aligned(1024))) char s_v[2][Tile::kBytes];
    __shared__ uint32_t s_last;
    __shared__ int s_odd;

    const int tid = threadIdx.x, lane = lane_id(), wave = wave_index();
    const int col = lane & 31, half = lane >> 5;
    PromptArgs &a = prompt_args();

    // The length as the caller counts it: a table that is too short hides
    // positions (n_seen), it does not move the new tokens.
    typedef __attribute__((address_space(4))) const int32_t const_i32;
    struct Seq {
        int tok0, n_new, n, tiles;
    };
    auto seq_of = [&](int b) {
        Seq x;
        x.tok0 = min(max((int)((const_i32 *)(uintptr_t)a.cu)[b], 0), a.tokens);
        x.n_new = min(max((int)((const_i32 *)(uintptr_t)a.cu)[b + 1], x.tok0), a.tokens) - x.tok0;
        x.n = max((int)((const_i32 *)(uintptr_t)a.lengths)[b], 0);
        x.tiles = row_tiles(x.n_new, a.group);
        return x;
    };
    const int most = a.cols << a.page_log2;
    // Tiles of keys that some row of a row tile sees.
    auto visible_of = [&](const Seq &x, int row0) {
        const int rows = min(kPromptRows, x.n_new * a.group - row0), past = x.n - x.n_new;
        const int lo = past + row0 / a.group, hi = past + (row0 + rows - 1) / a.group;
        // (Rows before the first position see nothing: they must not move the window
        // over the ends of an integer.)
        return visible<6>(max(0, min(min(x.n, most), hi + 1)),
                          a.window > 0 ? max(0, max(lo, 0) - a.window + 1) : 0, a.sinks);
    };

    // Equal shares: workgroups go round the XCDs, so neighbours in the sequence,
    // which read the same keys, are given to the workgroups of one of them.
    int h = (int)blockIdx.x % a.kv_heads, unit = (int)blockIdx.x / a.kv_heads;
    if (a.units) {
        const int xcd = (int)blockIdx.x & 7, per = (int)gridDim.x >> 3, more = (int)gridDim.x & 7;
        const int id = xcd * per + min(xcd, more) + ((int)blockIdx.x >> 3);
        h = id / a.units;
        unit = id - h * a.units;
    }
    int b = -1, tile = 0, index = 0;   // the row tile, and its place among all
    Seq seq = {};
    int64_t chunk = 0, at = 0, x0 = 0, x1 = 0;
    if (a.units == 0) {
        // One row tile, or a part of one: unit = tile * split + part.
        index = unit / a.split;
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
            const int first = base + wave_excl_scan(mine, &all);
            const uint64_t found = __ballot(index >= first && index < first + mine);
            if (found) {
                const int l = __builtin_ctzll(found);
                b = b0 + l;
                seq = seq_of(b);
                // late rows, which see most, first
                tile = seq.tiles - 1 - (index - __builtin_amdgcn_readlane(first, l));
                break;
            }
            base += (int)uniform(all);
        }
        if (b < 0) return;
    } else {
        // Equal shares of all tiles of keys, laid end to end; a row tile that
        // sees nothing counts as one.
        int64_t sum = 0;
        for (int bb = 0; bb < a.batch; ++bb) {
            const Seq x = seq_of(bb);
            for (int t = lane; t < x.tiles; t += 64)
                sum += kPromptFixed + max(1, visible_of(x, t * kPromptRows).total);
        }
#pragma unroll
        for (int y = 32; y >= 1; y >>= 1) sum += __shfl_xor(sum, y);
        sum = (int64_t)((uint64_t)uniform((uint32_t)(sum >> 32)) << 32 | uniform((uint32_t)sum));
        chunk = max((int64_t)kPromptLeast, (sum + a.units - 1) / a.units);
        x0 = unit * chunk;
        x1 = min(sum, x0 + chunk);
        if (x0 >= x1) return;
        for (int bb = 0; b < 0 && bb < a.batch; ++bb) {
            const Seq x = seq_of(bb);
            for (int t0 = 0; t0 < x.tiles; t0 += 64) {
                const int t = t0 + lane;
                const int w =
                    t < x.tiles ? kPromptFixed + max(1, visible_of(x, t * kPromptRows).total) : 0;
                int all;
                const int64_t first = at + wave_excl_scan(w, &all);
                const uint64_t found = __ballot(x0 >= first && x0 < first + w);
                if (found) {
                    const int l = __builtin_ctzll(found);
                    b = bb;
                    seq = x;
                    tile = t0 + l;
                    at += (int)uniform(__shfl((int)(first - at), l));
                    break;
                }
                at += (int)uniform(all);
            }
            index += b < 0 ? x.tiles : tile;
        }
        if (b < 0) return;
    }
    for (;;) {
        PromptArgs &a = prompt_args();
        // More than the tokens make up: a cu that decreases counts rows twice.
        if (index >= a.row_tiles) return;
        const int n_new = seq.n_new, tok0 = seq.tok0;
        const int n_seen = min(seq.n, most);
        const int row0 = tile * kPromptRows;
        const int rows = min(kPromptRows, n_new * a.group - row0);
        const int past = seq.n - n_new;
        const int pos_lo = past + row0 / a.group, pos_hi = past + (row0 + rows - 1) / a.group;
        const Visible vis = visible_of(seq, row0);
        // This workgroup's share of it, and where the parts of a split one go.
        constexpr int64_t kSlot = kPromptRows * (D + 2);
        int i0, i1, parts, part;
        int64_t slot0, weight = kPromptFixed + max(1, vis.total);
        if (a.units == 0) {
            const int c = max(1, (vis.total + a.split - 1) / a.split);
            parts = max(1, (vis.total + c - 1) / c);
            part = unit % a.split;
            if (part >= parts) return;
            i0 = part * c;
            i1 = min(vis.total, i0 + c);
            slot0 = ((int64_t)index * a.split * a.kv_heads + h) * kSlot;
        } else {
            const int64_t tiles_at = at + kPromptFixed;
            if (tiles_at >= x1) return;
            i0 = (int)(max(x0, tiles_at) - tiles_at);
            i1 = min(vis.total, (int)(min(x1, at + weight) - tiles_at));
            const int64_t first = tiles_at / chunk;
            parts = (int)((at + weight - 1) / chunk - first) + 1;
            part = (int)(unit - first);
            // A unit has at most two parts of split row tiles: one that began
            // before it, in its first slot, and one that goes on after it.
            slot0 = (first * 2 * a.kv_heads + h) * kSlot;
        }
        // This lane's row.
        const int my = row0 + min(32 * wave + col, rows - 1);
        const int my_tok = my / a.group, pos = past + my_tok;
        const int from = a.window > 0 ? max(pos, -1) - a.window : -1;   // sees keys above it
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

        const int32_t *table = a.tables + (int64_t)b * a.cols;
        constexpr int ES = F8 ? 1 : 2;
        const uint32_t head_bytes = D * ES << a.page_log2, page_bytes = head_bytes * a.kv_heads;
        const char *k_head = (const char *)a.k + (int64_t)h * head_bytes;
        const char *v_head = (const char *)a.v + (int64_t)h * head_bytes;
        const int in_page = (1 << a.page_log2) - 1;
        // Page numbers come by scalar loads (the tables are not written here): they
        // wait for nothing of the vector memory.
        const_i32 *table_c = (const_i32 *)(uintptr_t)table;
        auto page_of = [&](int key) {
            return (uint32_t)table_c[min(key >> a.page_log2, a.cols - 1)];
        };
        // Whether all positions of the share have a page: looked up once, since as a
        // rule they do.
        bool paged = true;
        for (int x = 4 * i0 + lane; x < 4 * i1; x += 64) {
            const int key = 64 * visible_block(vis, x >> 2) + 16 * (x & 3);
            paged &= key >= n_seen || (uint32_t)table[key >> a.page_log2] < (uint32_t)a.pages;
        }
        paged = __all(paged);
        // Wave w brings the 16 keys 16w .. 16w + 15 of a tile, which share a page:
        // where they start, in bytes of a head.
        auto offset_of = [&](int i) {
            const int key = (int)uniform(64 * visible_block(vis, i) + 16 * wave);
            uint32_t p = page_of(key);
            p = p < (uint32_t)a.pages ? p : 0u;
            return (uint64_t)p * page_bytes + (uint32_t)((key & in_page) * (D * ES));
        };
        // Rows x RPI .. of a wave's share, and the piece a lane brings of them.  Where
        // rows are as long in memory as in LDS, one base serves four pieces.
        constexpr int RPI = 64 / Tile::kSlots, CP = 16 / RPI;
        constexpr bool kSame = 2 * D == Tile::kRowBytes;
        constexpr int PN = !kSame ? 1 : CP < 4 ? CP : 4;
        uint32_t copy_off[F8 ? 1 : CP];
        if constexpr (!F8) {
#pragma unroll
            for (int x = 0; x < CP; ++x) {
                const int r = RPI * x + lane / Tile::kSlots;
                const int ch = (lane % Tile::kSlots) ^ Tile::swizzle(r);
                copy_off[x] = ch < Tile::kChunks ? r * (2 * D) + 16 * ch - 1024 * (x % PN) : ~0u;
            }
        }
        auto copy_in = [&](const char *head, const char *dst, uint64_t off) {
            const uint32_t to = uniform(lds_address(dst) + 16 * wave * Tile::kRowBytes);
#pragma unroll
            for (int x = 0; x < CP; x += PN) {
                if (Tile::kSlots == Tile::kChunks || copy_off[x] != ~0u)
                    copy_to_lds<PN>(head + off, copy_off + x, to + RPI * x * Tile::kRowBytes);
            }
        };
        // e4m3: a lane's share of 16 rows is 16 D / 64 codes, in chunks of 8.
        constexpr int NC = F8 ? D / 32 : 1;
        u32x2 raw_k[NC], raw_v[NC];
        auto fetch = [&](const char *head, u32x2 *raw, uint64_t off) {
            const char *src = head + off;
#pragma unroll
            for (int x = 0; x < NC; ++x) raw[x] = *(const u32x2 *)(src + 8 * (64 * x + lane));
        };
        auto convert = [&](const u32x2 *raw, char *dst) {
#pragma unroll
            for (int x = 0; x < NC; ++x) {
                const int r = (64 * x + lane) / Tile::kChunks, ch = (64 * x + lane) % Tile::kChunks;
                *(u32x4 *)(dst + Tile::byte_of(16 * wave + r, ch)) =
                    (u32x4){T::template from_e4m3<false>(raw[x][0]),
                            T::template from_e4m3<true>(raw[x][0]),
                            T::template from_e4m3<false>(raw[x][1]),
                            T::template from_e4m3<true>(raw[x][1])};
            }
        };

        f32x16 o[DT];
#pragma unroll
        for (int j = 0; j < DT; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[j][r] = 0.f;
        float m = kNoMax, l = 0.f;
        bool large = false;   // some row's maximum is

        // Where this lane reads, in bytes of a tile (tiles start at multiples of
        // 1024, so what follows holds for addresses, too).  Chunks of one row differ in
        // address bits of their own (the swizzle depends on the low bits of the row
        // alone), so operand j of K sits at (at_k ^ 32 j), and rows 32 further on at
        // a constant distance.  V is read transposed: a lane group of 16 brings keys
        // k0 .. k0 + 3 (k0 = 16 t + 4 half) of 16 columns, then the same 8 keys on.
        const int key_v = 4 * half + ((lane & 15) >> 2);
        const int dim_v = 16 * (lane >> 4 & 1) + 4 * (lane & 3);
        const uint32_t at_k = Tile::byte_of(col, half);
        const uint32_t at_v = Tile::byte_of(key_v, dim_v >> 3) + 2 * (dim_v & 7);
        auto v_op = [&](uint32_t at, int t, int dt) {  // at: at_v in a tile
            const uint32_t row = 16 * t * Tile::kRowBytes;
            const u32x2 x = read_transposed((at ^ 64 * dt) + row);
            const u32x2 y = read_transposed((at ^ (64 * dt ^ 32)) + row + 8 * Tile::kRowBytes);
            return (u32x4){x[0], x[1], y[0], y[1]};
        };

        // What rows see of a tile: which groups of 16 keys have a page, and whether
        // every row sees all of it.
        struct Seen {
            int key0;
            uint32_t have;
            bool whole;
        };
        const int whole_to = min(pos_lo - 63, n_seen - 64);
        const int whole_from = a.window > 0 ? max(pos_hi, 0) - a.window + 1 : 0;
        auto seen_of = [&](int i) {
            Seen x;
            x.key0 = (int)uniform(64 * visible_block(vis, i));
            x.have = 15;
            if (!paged) {
                x.have = 0;
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    x.have |= page_of(x.key0 + 16 * y) < (uint32_t)a.pages ? 1u << y : 0u;
            }
            x.whole = x.have == 15u && x.key0 <= whole_to &&
                      (x.key0 >= whole_from || x.key0 + 64 <= a.sinks);
            return x;
        };
        // Scores: keys down (2 x 32), rows across.  Operands are read four at a
        // time, one round ahead of the products that take them.
        auto scores = [&](const char *sk, f32x16 *s) {
            // Opaque, so that the operands' addresses are formed where they are
            // used: kept from tile to tile they take some forty registers.
            uint32_t ak = lds_address(sk) + at_k;
            asm("" : "+v"(ak));
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int r = 0; r < 16; ++r) s[u][r] = 0.f;
            u32x4 kb[2][4];
            auto read_k = [&](u32x4 *d, int f0) {
#pragma unroll
                for (int f = 0; f < 4; ++f)
                    d[f] = read_lds16((ak ^ 32 * ((f0 + f) >> 1)) +
                                      32 * ((f0 + f) & 1) * Tile::kRowBytes);
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
        // Values that no row sees become zero, and so do those that are not finite: a
        // row that does not see them would get NaN from them.  What they mean for the
        // rows that do see them comes at the end.
        auto clean = [&](const Seen &see, char *sv) {
            constexpr int N = kPromptKeys * Tile::kChunks / kPromptThreads;
            constexpr uint32_t exp2x = T::kOne == 0x3F80u ? 0x7F807F80u : 0x7C007C00u;
            constexpr uint32_t one2x = T::kOne == 0x3F80u ? 0x00800080u : 0x04000400u;
            int x0 = tid;  // opaque, as in scores()
            asm("" : "+v"(x0));
            u32x4 v[N];
#pragma unroll
            for (int y = 0; y < N; ++y) {
                const int x = x0 + kPromptThreads * y, r = x / Tile::kChunks;
                v[y] = ld16(sv + Tile::byte_of(r, x % Tile::kChunks));
            }
#pragma unroll
            for (int y = 0; y < N; ++y) {
                const int x = x0 + kPromptThreads * y, r = x / Tile::kChunks;
                u32x4 *p = (u32x4 *)(sv + Tile::byte_of(r, x % Tile::kChunks));
                uint32_t odd = 0;
#pragma unroll
                for (int z = 0; z < 4; ++z) odd |= (v[y][z] & exp2x) + one2x;
                const bool seen = see.key0 + r < n_seen && (see.have >> (r >> 4) & 1);
                if (!seen) {
                    *p = (u32x4){0, 0, 0, 0};
                } else if (odd & 0x80008000u) {
                    s_odd = 1;
#pragma unroll
                    for (int z = 0; z < 4; ++z) v[y][z] = finite_of<T>(v[y][z]);
                    *p = v[y];
                }
            }
            __syncthreads();
        };
        auto hide = [&](const Seen &see, f32x16 *s) {
            int key0 = see.key0 + 4 * half;  // opaque, as above
            asm("" : "+v"(key0));
            if (see.have == 15u && (a.window <= 0 || see.key0 >= a.sinks)) {
                // One run of keys: those from first on, and fewer than count of them.
                const int count = max(0, min(pos, n_seen - 1) - from);
                const uint32_t first = (uint32_t)key0 - (uint32_t)from - 1u;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        s[u][r] = first + (32 * u + 8 * (r >> 2) + (r & 3)) < (uint32_t)count
                                      ? s[u][r]
                                      : hidden;
                return;
            }
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

        __syncthreads();  // the LDS of the row tile before this one is free
        if (tid == 0) s_odd = 0;
        uint64_t next = 0;
        if (i0 < i1) {
            const uint64_t first = offset_of(i0);
            if constexpr (F8) {
                fetch(k_head, raw_k, first);
                fetch(v_head, raw_v, first);
                convert(raw_k, s_k[0]);
                convert(raw_v, s_v[0]);
            } else {
                copy_in(k_head, s_k[0], first);
                copy_in(v_head, s_v[0], first);
            }
            next = offset_of(min(i0 + 1, i1 - 1));
        }
        for (int i = i0; i < i1; ++i) {
            const int buf = (i - i0) & 1;
            char *sk = s_k[buf], *sv = s_v[buf];
            wait_vm_all();
            __syncthreads();  // this tile is here, and the other buffer is free
            const bool more = i + 1 < i1;
            if (more) {
                if constexpr (F8) {
                    fetch(k_head, raw_k, next);
                    fetch(v_head, raw_v, next);
                } else {
                    copy_in(k_head, s_k[buf ^ 1], next);
                    copy_in(v_head, s_v[buf ^ 1], next);
                }
            }
            const Seen see = seen_of(i);
            if (!see.whole) clean(see, sv);
            f32x16 s[2];
            scores(sk, s);
            uint32_t av = lds_address(sv) + at_v;
            asm("" : "+v"(av));
            u32x4 vb[2][4];
            auto read_v = [&](u32x4 *d, int f0) {
#pragma unroll
                for (int f = 0; f < 4; ++f) d[f] = v_op(av, (f0 + f) / DT, (f0 + f) % DT);
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
                large = __any(fabsf(m) > kLargeMax && m > kNoMax);
                l *= f;
#pragma unroll
                for (int j = 0; j < DT; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r) o[j][r] *= f;
            }
            u32x4 p[4];
            float by = c2, shift = T::kOff - m;
            if (large) {
#pragma clang fp contract(off)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[u][r] = s[u][r] * c2 - m;
                by = 1.f;
                shift = T::kOff;
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int r = 0; r < 16; r += 2) {
                    const float p0 = exp2_(fmaf(s[u][r], by, shift));
                    const float p1 = exp2_(fmaf(s[u][r + 1], by, shift));
                    // Weights are rounded to 16 bits for the second product (their
                    // sum is not): the output's error grows from 0.0016 to 0.0022
                    // in bf16.  The pair that decode uses would double that
                    // product, which with the first takes 45% of the time.
                    l += p0 + p1;
                    p[2 * u + (r >> 3)][(r & 7) >> 1] = T::pack(p0, p1);
                }
#pragma unroll
            for (int f = 0; f < 4 * DT; f += 4) {
                if (f + 4 < 4 * DT) read_v(vb[f / 4 + 1 & 1], f + 4);
                __builtin_amdgcn_sched_barrier(0);
                // Waves that are here go first: their operands are at hand.
                __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int t = (f + x) / DT, dt = (f + x) % DT;
                    o[dt] = T::mfma32(vb[f / 4 & 1][x], p[t], o[dt]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            __builtin_amdgcn_s_setprio(0);
            // Here, since behind a scalar load every wait for LDS is one for all of it.
            next = offset_of(min(i + 2, i1 - 1));
            if constexpr (F8) {
                if (more) {
                    convert(raw_k, s_k[buf ^ 1]);
                    convert(raw_v, s_v[buf ^ 1]);
                }
            }
        }
        float zero = 0.f;   // or NaN
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
            for (int r = 0; r < 16; ++r) zero = fmaf(o[dt][r], 0.f, zero);
        if (__any(zero != zero) && lane == 0) s_odd = 1;
        __syncthreads();
        const bool odd = s_odd;
        l += __shfl_xor(l, 32);

        PromptArgs &z = prompt_args();
        // Part k's slot; of equal shares, part 0 has the second slot of its unit.
        auto slot_of = [&](int k) {
            if (z.units == 0) return z.part + slot0 + (int64_t)k * z.kv_heads * kSlot;
            return z.part + slot0 + (int64_t)(k == 0 ? 1 : 2 * k) * z.kv_heads * kSlot;
        };
        const bool real = 32 * wave + col < rows;
        uint16_t *op = (uint16_t *)z.out + out_row * D;
        auto write = [&]() {
            const float f = l != 0.f ? (F8 && z.v_scale ? z.v_scale[h] : 1.f) / l : 0.f;
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
                z.lse[out_row] = l != 0.f ? (m + log2_(l) - T::kOff) * kLn2 : -__builtin_inff();
        };
        // Parts are kept as the lanes hold them (the one that joins them has
        // the same rows in the same places): every access is a whole block.
        const uint32_t at_part = 4u * (wave * 32 * (D + 2));
        if (parts > 1) {
            const rsrc_t to = buf_rsrc(slot_of(part));
#pragma unroll
            for (int dt = 0; dt < DT; ++dt)
#pragma unroll
                for (int r = 0; r < 16; r += 4) {
                    const f32x4 x = {o[dt][r], o[dt][r + 1], o[dt][r + 2], o[dt][r + 3]};
                    buf_st16<true>(to, at_part + 1024 * (4 * dt + r / 4) + 16 * lane,
                                   __builtin_bit_cast(u32x4, x));
                }
            float *ml = slot_of(part) + wave * 32 * (D + 2) + 32 * D + col;
            if (half == 0) {
                store_agent(ml, m);
                store_agent(ml + 32, l);
            }
        } else if (real) {
            write();
        }
        if (odd) {
            // Values that are not finite: a row's sum is the infinity (for NaN both)
            // of all that it sees.  The products leave that out where tiles were
            // cleaned, and make NaN of it where a weight or a factor is too small
            // for its type.  Rare, so values are brought again, 32 dimensions at a
            // time, and what was just written is written over.
            wait_vm_all();
            float *slot = slot_of(part) + wave * 32 * (D + 2) + 4 * lane;
#pragma unroll 1
            for (int dt = 0; dt < DT; ++dt) {
                f32x16 x[2];   // how many of +inf and NaN, and of -inf and NaN
#pragma unroll
                for (int r = 0; r < 16; ++r) x[0][r] = x[1][r] = 0.f;
#pragma unroll 1
                for (int i = i0; i < i1; ++i) {
                    const Seen see = seen_of(i);
                    const uint64_t off = offset_of(i);
                    __syncthreads();
                    if constexpr (F8) {
                        fetch(v_head, raw_v, off);
                        convert(raw_v, s_v[0]);
                    } else {
                        copy_in(v_head, s_v[0], off);
                    }
                    wait_vm_all();
                    __syncthreads();
                    f32x16 s[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int r = 0; r < 16; ++r) s[u][r] = 0.f;
                    if (!see.whole) hide(see, s);
                    u32x4 p[4];   // one for what the row sees
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int r = 0; r < 16; r += 2)
                            p[2 * u + (r >> 3)][(r & 7) >> 1] =
                                (s[u][r] == 0.f ? T::kOne : 0u) |
                                (s[u][r + 1] == 0.f ? T::kOne << 16 : 0u);
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const u32x4 v = v_op(lds_address(s_v[0]) + at_v, t, dt);
#pragma unroll
                        for (int sign = 0; sign < 2; ++sign) {
                            u32x4 marks;
#pragma unroll
                            for (int y = 0; y < 4; ++y) marks[y] = marks_of<T>(v[y], sign);
                            x[sign] = T::mfma32(marks, p[t], x[sign]);
                        }
                    }
                }
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    // (A row whose scores are not finite keeps its NaN.)
                    if ((x[0][r] == 0.f && x[1][r] == 0.f) || l != l) continue;
                    const float sum = sum_of_marks(x[0][r] != 0.f, x[1][r] != 0.f);
                    if (parts > 1)
                        store_agent(slot + 1024 * dt + 256 * (r / 4) + r % 4, sum);
                    else if (real)
                        op[32 * dt + 2 * (r & 12) + 4 * half + r % 4] =
                            (uint16_t)T::pack(F8 && z.v_scale ? sum * z.v_scale[h] : sum, 0.f);
                }
            }
        }
        if (parts > 1) {
            const int64_t group = (int64_t)index * z.kv_heads + h;
            wait_vm_all();
            __syncthreads();
            if (tid == 0)
                s_last = __hip_atomic_fetch_add(z.counters + group, 1u, __ATOMIC_RELAXED,
                                                __HIP_MEMORY_SCOPE_AGENT);
            __syncthreads();
            if (s_last == (uint32_t)parts - 1) {
                if (tid == 0) store_agent(z.counters + group, 0u);
                // Loads of several parts are on their way together: one after
                // the other they cost most of a microsecond each.
                const int ml = wave * 32 * (D + 2) + 32 * D + col;
                m = kNoMax;
                for (int k = 0; k < parts; k += 8) {
                    float x[8];
#pragma unroll
                    for (int y = 0; y < 8; ++y) x[y] = load_agent(slot_of(min(k + y, parts - 1)) + ml);
#pragma unroll
                    for (int y = 0; y < 8; ++y) m = fmaxf(m, x[y]);
                }
                l = 0.f;
#pragma unroll
                for (int dt = 0; dt < DT; ++dt)
#pragma unroll
                    for (int r = 0; r < 16; ++r) o[dt][r] = 0.f;
                constexpr int K = DT <= 4 ? 2 : 1;   // parts at a time
                for (int k = 0; k < parts; k += K) {
                    float pm[K], pl[K];
                    f32x4 x[K][4 * DT];
#pragma unroll
                    for (int y = 0; y < K; ++y) {
                        const float *slot = slot_of(min(k + y, parts - 1));
                        const rsrc_t of = buf_rsrc(slot);
                        pm[y] = load_agent(slot + ml);
                        pl[y] = load_agent(slot + ml + 32);
#pragma unroll
                        for (int z = 0; z < 4 * DT; ++z)
                            x[y][z] = __builtin_bit_cast(
                                f32x4, buf_ld16<true>(of, at_part + 1024 * z + 16 * lane));
                    }
#pragma unroll
                    for (int y = 0; y < K; ++y) {
                        const float f = k + y < parts ? part_factor(pm[y] - m) : 0.f;
                        l = fmaf(pl[y], f, l);
#pragma unroll
                        for (int z = 0; z < 4 * DT; ++z)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float sum = o[z >> 2][4 * (z & 3) + e];
                                o[z >> 2][4 * (z & 3) + e] =
                                    k + y < parts ? fmaf(x[y][z][e], f, sum) : sum;
                            }
                    }
                }
                if (real) write();
            }
        }
        // On to the next row tile of an equal share.
        at += weight;
        if (z.units == 0 || at >= x1) return;
        ++index;
        if (++tile == seq.tiles) {
            tile = 0;
            do {
                if (++b >= z.batch) return;
                seq = seq_of(b);
            } while (seq.tiles == 0);
        }
    }
}

}  // namespace serve
}  // namespace moe
