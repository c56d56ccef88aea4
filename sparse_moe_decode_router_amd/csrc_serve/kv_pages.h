// kv_pages.h - the upkeep of the paged cache: new keys and values into their
// pages, and the pages themselves (free, fork, extend, compact).
//
// The bookkeeping of a call (which pages are free, who gets them) is done by
// one workgroup: it is a scan over the pool's reference counts, 4096 of them a
// round, and the results have to be the lowest pages in a fixed order.  It is a
// chain of dependent loads (fork of 32 pairs 6.5 us, compact of 1100 pages 6.0);
// more workgroups would have to wait for each other several times.  The pages'
// contents are moved by a second launch over the whole chip, bound by memory
// (282 pages of 1 MB over 4 layers: 121 us, 4.9 TB/s).
#pragma once

#include "serve_common.h"
#include "moe_serve.h"

namespace moe {
namespace serve {

struct AppendArgs {
    const void *k, *v;
    void *kc, *vc;             // the layer's pages
    const int32_t *tables, *lengths, *cu;
    const int32_t *granted;    // or NULL: positions that a sequence was given
    const float *k_scale, *v_scale;
    int64_t token_stride, head_stride;
    int32_t tokens, batch, pages, cols, page_log2, kv_heads, head_dim;
    int32_t per_block;         // tokens a workgroup takes
};

// Eight values -> eight e4m3 codes of x / scale.  The division is the IEEE one
// (a reciprocal could move a value over a rounding border); the clamp keeps NaN.
template <class T>
__device__ __forceinline__ u32x2 to_e4m3(u32x4 x, float scale) {
    uint32_t r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float f[4] = {T::lo(x[2 * i]), T::hi(x[2 * i]), T::lo(x[2 * i + 1]), T::hi(x[2 * i + 1])};
        uint32_t nan = 0, sign = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[j] = f[j] / scale;
            nan |= f[j] != f[j] ? 0xFFu << 8 * j : 0u;
            sign |= __float_as_uint(f[j]) >> 31 << (8 * j + 7);
            f[j] = fminf(fmaxf(f[j], -448.f), 448.f);
        }
        uint32_t w = 0;
        w = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], w, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], w, true);
        r[i] = (w & ~nan) | (nan & (0x7F7F7F7Fu | sign));
    }
    return (u32x2){r[0], r[1]};
}

// A workgroup takes `per_block` consecutive tokens, a thread chunks of eight
// elements of one head's row (keys and values).  The first token's sequence is
// found by bisection with uniform loads, later ones from there.  Bound by memory:
// 20750 tokens of 8 heads of 128 in bf16, 170 MB, take 37 us (4.6 TB/s); one
// token of 64 sequences takes 3.3 us, most of it the launch.
template <class T, bool F8>
__global__ __launch_bounds__(256) void k_kv_append(const AppendArgs a) {
    const int t0 = (int)blockIdx.x * a.per_block;
    const int t1 = min(t0 + a.per_block, a.tokens);
    int b0 = t0;
    if (a.cu) {
        int lo = 0, hi = a.batch;  // the last b with cu[b] <= t0
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.cu[mid] <= t0) lo = mid;
            else hi = mid;
        }
        b0 = lo;
    }
    const int per_head = a.head_dim >> 3, per_token = per_head * a.kv_heads;
    const int most = a.cols << a.page_log2;
    for (int x = threadIdx.x; x < (t1 - t0) * per_token; x += 256) {
        const int t = t0 + x / per_token, ch = x % per_token;
        int b = t, pos, n_new = 1;
        if (a.cu) {
            b = b0;
            while (b + 1 < a.batch && a.cu[b + 1] <= t) ++b;
            if (t < a.cu[b] || t >= a.cu[b + 1]) continue;
            n_new = a.cu[b + 1] - a.cu[b];
            pos = a.lengths[b] - (a.cu[b + 1] - t);
        } else {
            pos = a.lengths[b] - 1;
        }
        if (pos < 0 || pos >= most || (a.granted && a.granted[b] < n_new)) continue;
        const uint32_t page = (uint32_t)a.tables[(int64_t)b * a.cols + (pos >> a.page_log2)];
        if (page >= (uint32_t)a.pages) continue;
        const int h = ch / per_head, d = 8 * (ch % per_head);
        const int64_t from = t * a.token_stride + h * a.head_stride + d;
        const int64_t to =
            ((((int64_t)page * a.kv_heads + h) << a.page_log2) + (pos & ((1 << a.page_log2) - 1))) *
                a.head_dim + d;
        const u32x4 k = ld16((const uint16_t *)a.k + from), v = ld16((const uint16_t *)a.v + from);
        if constexpr (F8) {
            *(u32x2 *)((uint8_t *)a.kc + to) = to_e4m3<T>(k, a.k_scale ? a.k_scale[h] : 1.f);
            *(u32x2 *)((uint8_t *)a.vc + to) = to_e4m3<T>(v, a.v_scale ? a.v_scale[h] : 1.f);
        } else {
            *(u32x4 *)((uint16_t *)a.kc + to) = k;
            *(u32x4 *)((uint16_t *)a.vc + to) = v;
        }
    }
}

// ---- Bookkeeping -----------------------------------------------------------

struct PagesArgs {
    int32_t *tables, *lengths, *refs;
    uint32_t *flags;
    const int32_t *from, *to;      // fork: parents, children; extend / free: from = seqs
    const int32_t *counts;         // extend
    int32_t *granted;              // extend: by sequence, or NULL
    int32_t *new_tables, *new_refs;  // compact
    int32_t *scratch;
    int32_t n, pages, page_log2, seqs, cols;
};

constexpr int kPagesThreads = 1024;
constexpr int kPagesWaves = kPagesThreads / 64;

// Scratch of fork: [0] pairs to copy, then (source, target) per pair (-1: none);
// before that (rank among those that need a page, or -1: no last page in part, -2:
// a missing one; length).  Of
// extend and fork also the list of pages taken, from `list` on.  Of compact:
// [0] pages to move, then the targets, the sources, and each page's new place.
constexpr int kScratchHead = 4;

// Exclusive prefix sum of v over the workgroup; *total: the sum.
__device__ __forceinline__ int block_scan(int v, int *total, int *s_wave) {
    const int lane = lane_id(), wave = wave_index();
    int all;
    const int at = wave_excl_scan(v, &all);
    __syncthreads();
    if (lane == 0) s_wave[wave] = all;
    __syncthreads();
    int before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kPagesWaves; ++w) {
        const int x = s_wave[w];
        before += w < wave ? x : 0;
        sum += x;
    }
    *total = sum;
    return before + at;
}

// Writes the lowest `want` pages p with test(p) into list; returns how many
// there were (at most want).
template <class Test>
__device__ __forceinline__ int take_lowest(int pages, int want, int32_t *list, int *s_wave,
                                           Test test) {
    int found = 0;
    for (int p0 = 0; p0 < pages && found < want; p0 += 4 * kPagesThreads) {
        const int p = p0 + 4 * (int)threadIdx.x;
        uint32_t hit = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (p + i < pages && test(p + i)) hit |= 1u << i;
        int all, at = found + block_scan(__popc(hit), &all, s_wave);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (hit >> i & 1) {
                if (at < want) list[at] = p + i;
                ++at;
            }
        found += all;
    }
    return min(found, want);
}

__global__ __launch_bounds__(256) void k_kv_free(const PagesArgs a) {
    for (int x = blockIdx.x; x < a.n; x += gridDim.x) {
        const int s = a.from[x];
        if (s < 0 || s >= a.seqs) continue;
        int32_t *row = a.tables + (int64_t)s * a.cols;
        for (int i = threadIdx.x; i < a.cols; i += 256) {
            const int p = row[i];
            if (p >= 0) {
                if (p < a.pages) atomicAdd(a.refs + p, -1);
                row[i] = -1;
            }
        }
        if (threadIdx.x == 0) a.lengths[s] = 0;
    }
}

// Length of sequence s, cut to its table; 0 for one the cache does not have.
__device__ __forceinline__ int length_of(const PagesArgs &a, int s) {
    return s >= 0 && s < a.seqs ? min(max(a.lengths[s], 0), a.cols << a.page_log2) : 0;
}

__global__ __launch_bounds__(kPagesThreads) void k_kv_fork(const PagesArgs a) {
    __shared__ int s_wave[kPagesWaves];
    const int tid = threadIdx.x, page = 1 << a.page_log2;
    int32_t *copies = a.scratch + kScratchHead, *list = copies + 2 * a.n;
    // Which pairs need a page of their own, and their rank among those.
    int need = 0;
    for (int i0 = 0; i0 < a.n; i0 += kPagesThreads) {
        const int i = i0 + tid;
        const int len = i < a.n ? length_of(a, a.from[i]) : 0;
        const bool ok = i < a.n && a.to[i] >= 0 && a.to[i] < a.seqs;
        // A last page that the parent does not have needs no copy either.
        const int part = ok && (len & (page - 1)) &&
                                 (uint32_t)a.tables[(int64_t)a.from[i] * a.cols +
                                                    (len >> a.page_log2)] < (uint32_t)a.pages
                             ? 1
                             : 0;
        int all;
        const int at = need + block_scan(part, &all, s_wave);
        if (i < a.n) {  // the rank and the length, until pages are known
            copies[2 * i] = part ? at : len & (page - 1) ? -2 : -1;
            copies[2 * i + 1] = len;
        }
        need += all;
    }
    const int found = take_lowest(a.pages, need, list, s_wave, [&](int p) { return a.refs[p] == 0; });
    __syncthreads();
    if (tid == 0 && found < need) atomicOr(a.flags, (uint32_t)MOE_KV_FLAG_NO_PAGES);
    // Tables and references.  A pair's threads all read its rank and length
    // before the last loop replaces them.  (All counts fit 32 bits.)
    const uint32_t entries = (uint32_t)a.n * (uint32_t)a.cols;
    for (uint32_t x = tid; x < entries; x += kPagesThreads) {
        const int i = (int)(x / (uint32_t)a.cols), col = (int)(x % (uint32_t)a.cols);
        const int child = a.to[i], parent = a.from[i];
        const int rank = copies[2 * i], full = copies[2 * i + 1] >> a.page_log2;
        if (child < 0 || child >= a.seqs) continue;
        int p = -1;
        if (col < full) {
            p = a.tables[(int64_t)parent * a.cols + col];
            if (p >= 0 && p < a.pages) atomicAdd(a.refs + p, 1);
        } else if (col == full && rank >= 0 && rank < found) {
            p = list[rank];
            a.refs[p] = 1;
        } else if (col == full && rank == -2) {
            p = a.tables[(int64_t)parent * a.cols + col];  // not a page
        }
        a.tables[(int64_t)child * a.cols + col] = p;
    }
    __syncthreads();
    for (int i = tid; i < a.n; i += kPagesThreads) {
        const int child = a.to[i], rank = copies[2 * i], len = copies[2 * i + 1];
        const int full = len >> a.page_log2;
        int src = -1, dst = -1;
        if (rank >= 0 && rank < found) {
            src = a.tables[(int64_t)a.from[i] * a.cols + full];
            dst = list[rank];
        }
        copies[2 * i] = src;
        copies[2 * i + 1] = dst;
        if (child >= 0 && child < a.seqs)
            a.lengths[child] = rank >= 0 && rank >= found ? full << a.page_log2 : len;
    }
}

__global__ __launch_bounds__(kPagesThreads) void k_kv_extend(const PagesArgs a) {
    __shared__ int s_wave[kPagesWaves];
    const int tid = threadIdx.x, up = (1 << a.page_log2) - 1;
    int32_t *ranks = a.scratch + kScratchHead, *list = ranks + 2 * a.n;
    const int64_t most = (int64_t)a.cols << a.page_log2;
    auto seq = [&](int i) { return a.from ? a.from[i] : i; };
    int need = 0;
    for (int i0 = 0; i0 < a.n; i0 += kPagesThreads) {
        const int i = i0 + tid;
        int more = 0;
        if (i < a.n) {
            const int s = seq(i), len = length_of(a, s);
            const int64_t to = (int64_t)len + max(a.counts[i], 0);
            if (s >= 0 && s < a.seqs && to <= most)
                more = (int)((to + up) >> a.page_log2) - ((len + up) >> a.page_log2);
            else if (s >= 0 && s < a.seqs) {
                atomicOr(a.flags, (uint32_t)MOE_KV_FLAG_NO_COLS);
                if (a.granted) a.granted[s] = 0;
                more = -1;
            } else
                more = -1;
        }
        int all;
        const int at = need + block_scan(max(more, 0), &all, s_wave);
        if (i < a.n) {
            ranks[2 * i] = at;
            ranks[2 * i + 1] = more;
        }
        need += all;
    }
    const int want = min(need, a.pages);
    const int found = take_lowest(a.pages, want, list, s_wave, [&](int p) { return a.refs[p] == 0; });
    __syncthreads();
    if (found < need) {
        // Too few for all: in the order of the list, who does not find enough left
        // takes none.  Each choice depends on those before it, so one wave goes
        // through them, 64 in its registers at a time.
        for (int i0 = 0, used = 0; i0 < a.n && tid < 64; i0 += 64) {
            const int i = i0 + tid, more = i < a.n ? ranks[2 * i + 1] : -1;
            int at = 0;
            for (int j = 0; j < 64; ++j) {
                const int m = __builtin_amdgcn_readlane(more, j);
                const bool fits = m <= found - used;
                if (tid == j) at = fits ? used : -1;
                if (fits) used += max(m, 0);
            }
            if (i < a.n) ranks[2 * i] = at;
        }
        __syncthreads();
    }
    for (int i = tid; i < a.n; i += kPagesThreads) {
        const int at = ranks[2 * i], more = ranks[2 * i + 1];
        if (more < 0) continue;
        const int s = seq(i);
        if (more > 0 && at < 0) {
            atomicOr(a.flags, (uint32_t)MOE_KV_FLAG_NO_PAGES);
            if (a.granted) a.granted[s] = 0;
            continue;
        }
        const int len = length_of(a, s);
        const int col = (len + up) >> a.page_log2;
        for (int j = 0; j < more; ++j) {
            a.tables[(int64_t)s * a.cols + col + j] = list[at + j];
            a.refs[list[at + j]] = 1;
        }
        a.lengths[s] = len + max(a.counts[i], 0);
        if (a.granted) a.granted[s] = max(a.counts[i], 0);
    }
}

// Bookkeeping of compact: the live pages' new places.
__global__ __launch_bounds__(kPagesThreads) void k_kv_compact(const PagesArgs a) {
    __shared__ int s_wave[kPagesWaves];
    const int tid = threadIdx.x;
    int32_t *to = a.scratch + kScratchHead, *from = to + a.pages, *place = from + a.pages;
    int live = 0;
    for (int p = tid; p < a.pages; p += kPagesThreads) live += a.refs[p] > 0;
    int n_live;
    block_scan(live, &n_live, s_wave);
    // As many used pages lie from n_live on as free ones below it.
    int holes = 0, moved = 0;
    for (int p0 = 0; p0 < a.pages; p0 += kPagesThreads) {
        const int p = p0 + tid;
        const bool used = p < a.pages && a.refs[p] > 0;
        const bool hole = p < n_live && !used, move = p >= n_live && used;
        int all;
        // Both counts in one scan: a round has at most 1024 of each.
        const int at = block_scan((hole ? 1 : 0) | (move ? 1 << 16 : 0), &all, s_wave);
        if (hole) to[holes + (at & 0xFFFF)] = p;
        if (move) from[moved + (at >> 16)] = p;
        if (p < a.pages) place[p] = p;
        holes += all & 0xFFFF;
        moved += all >> 16;
    }
    __syncthreads();
    if (tid == 0) a.scratch[0] = moved;
    for (int i = tid; i < moved; i += kPagesThreads) place[from[i]] = to[i];
    // References: in place as well, so every round's reads (from n_live on)
    // come before anything there is cleared.
    if (a.new_refs != a.refs)
        for (int p = tid; p < n_live; p += kPagesThreads) a.new_refs[p] = a.refs[p];
    __syncthreads();
    for (int i = tid; i < moved; i += kPagesThreads) a.new_refs[to[i]] = a.refs[from[i]];
    __syncthreads();
    for (int p = n_live + tid; p < a.pages; p += kPagesThreads) a.new_refs[p] = 0;
}

// ---- Moving pages ----------------------------------------------------------

struct MoveArgs {
    char *data;
    int64_t plane_bytes, page_bytes;  // of one layer's keys or values; of one page
    int32_t planes;
    const int32_t *count;        // pages to move on the device, or NULL: n
    const int32_t *from, *to;    // stride apart
    int32_t stride, n, pages;
    // compact: the tables' new contents
    const int32_t *tables, *place;
    int32_t *new_tables;
    int64_t entries;
};

constexpr int kMoveChunk = 256 * 4 * 16;  // bytes a workgroup moves at a time

__global__ __launch_bounds__(256) void k_kv_move(const MoveArgs a) {
    const int tid = threadIdx.x;
    for (int64_t x = (int64_t)blockIdx.x * 256 + tid; x < a.entries; x += (int64_t)gridDim.x * 256) {
        const int p = a.tables[x];
        a.new_tables[x] = p >= 0 && p < a.pages ? a.place[p] : p;
    }
    const int n = a.count ? min(*a.count, a.n) : a.n;
    const int chunks = (int)((a.page_bytes + kMoveChunk - 1) / kMoveChunk);
    const int64_t all = (int64_t)n * a.planes * chunks;
    for (int64_t x = blockIdx.x; x < all; x += gridDim.x) {
        const int ch = (int)(x % chunks);
        const int64_t y = x / chunks;
        const int plane = (int)(y % a.planes), i = (int)(y / a.planes);
        const int src = a.from[(int64_t)i * a.stride], dst = a.to[(int64_t)i * a.stride];
        if (src < 0 || dst < 0) continue;
        const int64_t off = (int64_t)ch * kMoveChunk + 16 * tid;
        const char *s = a.data + plane * a.plane_bytes + src * a.page_bytes;
        char *d = a.data + plane * a.plane_bytes + dst * a.page_bytes;
        u32x4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (off + 4096 * j < a.page_bytes) v[j] = ld16(s + off + 4096 * j);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (off + 4096 * j < a.page_bytes) *(u32x4 *)(d + off + 4096 * j) = v[j];
    }
}

}  // namespace serve
}  // namespace moe
