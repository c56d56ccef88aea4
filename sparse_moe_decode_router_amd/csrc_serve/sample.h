// sample.h - the next tokens from rows of logits: temperature, top-k, top-p and
// min-p, and a given uniform number for each row.
//
// Weights are w = exp((x - max) / T).  Tokens are ordered by x, the largest first,
// equal ones by index; what the filters keep is a beginning of that order (and w >=
// min_p), and the token is the first in order of index at which the sum of the kept
// weights exceeds u times their sum.  Which token that is depends on sums over up
// to 2^19 weights next to borders that lie as close, so weights and sums are in 64
// bits; 32 would give another token every few hundred rows.
//
// Nothing is sorted as a whole.  A row is cut into slices, one workgroup each:
//   k_sample_scan   each slice's maximum and a histogram of its values over bins of
//                   1/64 in units of T ln 2: how many, and their weights to some
//                   20 bits, both in one 64-bit integer addition.  The last slice of
//                   a row finds the few bins in which the filters' borders are.
//   k_sample_draw   every slice sums, in 64 bits, the weights above those bins, and lists
//                   the values in them.  The last slice of a row to finish sorts
//                   that list, finds the border, the segment (a wave's share of a
//                   slice) that holds the token, and the token.
// Bins are monotonic in the value and their counts exact, so that the list holds the
// border whatever the weights' 20 bits missed (the margin of the search covers
// that).  Where the list would be too long (thousands of equal logits at the border),
// the last workgroup narrows the bins down by histograms of the values' bits instead,
// 11 bits a pass over the row.
//   k_sample_plain  rows without filters: each segment's maximum and sum, and the last
//                   slice draws.  One launch.
#pragma once

#include "serve_common.h"

namespace moe {
namespace serve {

constexpr int kSampleThreads = 512;
constexpr int kSampleWaves = kSampleThreads / 64;
constexpr int kSampleChunks = 32;       // most 16-byte chunks of a lane
constexpr int kSampleMaxSlices = 9;     // (2^19 values in 32 bits that begin inside a chunk)
constexpr int kSampleMaxDraws = 32;     // slices of k_sample_draw and k_sample_plain
constexpr int kSampleSegments = kSampleMaxDraws * kSampleWaves;
constexpr int kSampleBins = 4096;       // the last one takes all that is below
constexpr float kSamplePerOctave = 64.f;
constexpr int kSampleList = 4096;       // values at the border of a row
constexpr int kSampleKeyBins = 2048;    // of the values' bits
constexpr int kSampleSlots = 3;         // sums of a segment: above, above and kept, all

struct SampleSlice {
    float max;         // -inf: nothing to draw
    int32_t first;     // index of the first value that is the maximum
    int32_t bin;       // of the maximum
    int32_t count;     // finite values, and +inf
};

// What the slices of a row agree on: values from `top` on are kept by the filters, those
// below `bottom` are not, and the border is between (a NaN that nothing reaches: none).
struct SampleBorder {
    float top, bottom;
    int above, listed;    // values from top on, and from bottom to there
};

struct SampleArgs {
    const void *x;
    const float *u;
    const float *temperature, *top_p, *min_p;   // by row, or NULL: those for all
    const int32_t *top_k;
    float temperature_all, top_p_all, min_p_all;
    int32_t top_k_all;
    int32_t *token;
    float *logprob;
    SampleSlice *slices;      // [rows][slices]
    uint64_t *hist;           // [rows][slices][kSampleBins]: count << 44 | weights
    SampleBorder *borders;    // [rows]
    double *sums;             // [rows][draws][waves][kSampleSlots] (plain: the sum, the maximum)
    uint64_t *keys;           // [rows][draws][waves]: smallest and largest key of listed ones
    uint64_t *list;           // [rows][draws][kSampleList]
    int32_t *listed;          // [rows][draws]
    uint32_t *counters;       // [rows]: arrivals
    int64_t stride;           // of rows, in elements
    int32_t rows, vocab;
    int32_t slices_n;         // of k_sample_scan
    int32_t draws;            // of the others; sums, keys and lists are by them
    int32_t chunks, draw_chunks;   // of a wave's segment
};

enum { kSampleF32 = 3 };   // beside MOE_BF16 and MOE_FP16

__device__ __forceinline__ int max_i(int a, int b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t max_u(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The logits of a 16-byte chunk.
template <int Type>
struct Logits {
    static constexpr int kPer = Type == kSampleF32 ? 4 : 8;
    static constexpr int kBytes = 16 / kPer;
    static __device__ __forceinline__ float get(u32x4 c, int e) {
        if constexpr (Type == kSampleF32) return __uint_as_float(c[e]);
        if constexpr (Type == 0) return e & 1 ? Bf16::hi(c[e >> 1]) : Bf16::lo(c[e >> 1]);
        return e & 1 ? Fp16::hi(c[e >> 1]) : Fp16::lo(c[e >> 1]);
    }
    // Makes it -inf.
    static __device__ __forceinline__ void hide(u32x4 &c, int e) {
        if constexpr (Type == kSampleF32) {
            c[e] = 0xFF800000u;
        } else {
            const uint32_t h = Type == 0 ? 0xFF80u : 0xFC00u;
            c[e >> 1] = e & 1 ? (c[e >> 1] & 0xFFFFu) | h << 16 : (c[e >> 1] & 0xFFFF0000u) | h;
        }
    }
};

// A row's filters, as they act.
struct SampleRow {
    float temperature, top_p, min_p, u;
    int top_k;          // 0: off
    bool greedy, by_p;
};
__device__ __forceinline__ SampleRow sample_row(const SampleArgs &a, int row) {
    SampleRow r;
    const float t = a.temperature ? a.temperature[row] : a.temperature_all;
    r.greedy = !(t >= 0x1p-100f);               // zero, negative, NaN
    r.temperature = fminf(t, 0x1p100f);
    const int k = a.top_k ? a.top_k[row] : a.top_k_all;
    r.top_k = k > 0 && k < a.vocab ? k : 0;
    const float p = a.top_p ? a.top_p[row] : a.top_p_all;
    r.by_p = p < 1.f;
    r.top_p = fmaxf(p, 0.f);
    const float m = a.min_p ? a.min_p[row] : a.min_p_all;
    r.min_p = m > 0.f ? fminf(m, 1.f) : 0.f;
    const float u = a.u[row];
    r.u = u > 0.f ? fminf(u, 1.f) : 0.f;
    return r;
}

// A value's place in units of T ln 2 / 64, and its bin, the place rounded down: both
// monotonic in the value.  NaN has the place of -inf.
__device__ __forceinline__ float sample_scale(float temperature) {
    return fminf(kSamplePerOctave * kLog2e / temperature, 0x1p90f);
}
__device__ __forceinline__ float sample_place(float x, float scale) {
    return __builtin_amdgcn_fmed3f(x * scale, -0x1p29f, 0x1p29f);
}
__device__ __forceinline__ int sample_bin(float place) { return (int)__builtin_floorf(place); }
// The first bin of a slice or row: the maximum's, but never so low that -inf, whose place is
// the lowest, were not in the last one.
__device__ __forceinline__ int sample_top(float place) {
    return max_i(sample_bin(place), -(1 << 29) + 2 * kSampleBins);
}

// 2^y for y <= 1 (NaN: 0), to 2^-44: with r = y less the nearest integer, 1 + r q(r),
// where q has the values of (2^r - 1) / r at nine Chebyshev nodes of [-1/2, 1/2].
__device__ __forceinline__ double exp2_64(double y) {
    y = fmax(y, -1100.0);
    const double n = __builtin_rint(y), r = y - n;
    double q = 1.0203121063391729e-07;
    q = fma(q, r, 1.3255224878668817e-06);
    q = fma(q, r, 1.525268684626772e-05);
    q = fma(q, r, 0.00015403455852453838);
    q = fma(q, r, 0.0013333558179043112);
    q = fma(q, r, 0.009618129159402558);
    q = fma(q, r, 0.055504108664760424);
    q = fma(q, r, 0.2402265069581299);
    q = fma(q, r, 0.6931471805599453);
    return __builtin_ldexp(fma(q, r, 1.0), (int)n);
}
// c: log2(e) / T.  The maximum has weight 1, also where it is infinite; -inf and NaN
// have none.
__device__ __forceinline__ double sample_weight(float x, float max, double c) {
    if (max == __builtin_inff()) return x == max ? 1.0 : 0.0;
    return exp2_64(((double)x - (double)max) * c);
}

// Order of values as unsigned integers: larger x, smaller key.  NaN counts as -inf, and
// the two zeros are equal.
__device__ __forceinline__ uint32_t sample_key(float x) {
    const uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);
    return b >> 31 ? b : ~b & 0x7FFFFFFFu;
}
__device__ __forceinline__ float sample_value(uint32_t key) {
    return __uint_as_float(key >> 31 ? key : ~key & 0x7FFFFFFFu);
}

// Adds the value that DPP control `C` brings in the rows of `Rows`, elsewhere zero.
template <int C, int Rows, class V>
__device__ __forceinline__ V add_dpp(V v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, C, Rows, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), C, Rows, 0xF, false);
    return v + __builtin_bit_cast(V, (uint64_t)hi << 32 | lo);
}
// Sums (of 64 bits) up to and with each lane: within rows of 16, then from row to row.
template <class V>
__device__ __forceinline__ V wave_scan_d(V v) {
    v = add_dpp<0x111, 0xF>(v);     // from 1, 2, 4, 8 lanes below
    v = add_dpp<0x112, 0xF>(v);
    v = add_dpp<0x114, 0xF>(v);
    v = add_dpp<0x118, 0xF>(v);
    v = add_dpp<0x142, 0xA>(v);     // rows 1 and 3: the last lane of the row before
    return add_dpp<0x143, 0xC>(v);  // rows 2 and 3: lane 31
}
__device__ __forceinline__ double lane_d(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)b, lane);
    const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(b >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum_d(double v) { return lane_d(wave_scan_d(v), 63); }
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v = fmaxf(v, __shfl_xor(v, m));
    return v;
}
__device__ __forceinline__ int wave_min_i(int v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v = min(v, __shfl_xor(v, m));
    return v;
}
// Sum of the threads' values before this one, and of all.
template <class V>
__device__ __forceinline__ V block_scan_d(V v, V *total, V *s_wave) {
    const V inc = wave_scan_d(v);
    __syncthreads();
    if (lane_id() == 63) s_wave[wave_index()] = inc;
    __syncthreads();
    V before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kSampleWaves; ++w) {
        if (w < wave_index()) before += s_wave[w];
        all += s_wave[w];
    }
    *total = all;
    // (Not inc - v: the sum of what is before has its own rounding.)
    const uint64_t b = __builtin_bit_cast(uint64_t, inc);
    const uint32_t lo = __shfl_up((uint32_t)b, 1), hi = __shfl_up((uint32_t)(b >> 32), 1);
    return before + (lane_id() ? __builtin_bit_cast(V, (uint64_t)hi << 32 | lo) : (V)0);
}
__device__ __forceinline__ int block_scan_i(int v, int *total, int *s_wave) {
    int all;
    const int at = wave_excl_scan(v, &all);
    __syncthreads();
    if (lane_id() == 0) s_wave[wave_index()] = all;
    __syncthreads();
    int before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kSampleWaves; ++w) {
        if (w < wave_index()) before += s_wave[w];
        sum += s_wave[w];
    }
    *total = sum;
    return before + at;
}
__device__ __forceinline__ void store_agent_d(double *p, double v) {
    __hip_atomic_store((uint64_t *)p, __builtin_bit_cast(uint64_t, v), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ double load_agent_d(const double *p) {
    return __builtin_bit_cast(double, __hip_atomic_load((const uint64_t *)p, __ATOMIC_RELAXED,
                                                        __HIP_MEMORY_SCOPE_AGENT));
}

// A wave's segment: `chunks` 16-byte chunks from its first on, in the row's memory cut at
// multiples of 16 bytes, so that every load is aligned; values before the row's first and
// from `vocab` on are no values.
template <int Type>
struct Segment {
    typedef Logits<Type> L;
    const char *row;
    int shift;              // values before the row's first in its first chunk
    int chunk0, chunks;
    int total;              // chunks of the row

    __device__ __forceinline__ Segment(const SampleArgs &a, int r, int segment, int chunks)
        : chunks(chunks) {
        const uintptr_t at = (uintptr_t)a.x + (uint64_t)r * a.stride * L::kBytes;
        row = (const char *)at;
        shift = (int)(at & 15) / L::kBytes;
        chunk0 = segment * chunks;
        total = (shift + a.vocab + L::kPer - 1) / L::kPer;
    }
    // f(value, index) for every value of this lane (NaN too), as often in all lanes; what
    // is beyond the row is -inf.  Four values to a round of the loop: more of them are more
    // code than is fetched while a short segment's values are on their way (two thirds of
    // the time of one row went into that), and as many registers.
    template <class F>
    __device__ __forceinline__ void each(int vocab, F f) const {
        const char *base = row - shift * L::kBytes;
        const int lane = lane_id();
        auto load = [&](int i0) {
            return ld16(base + 16 * (int64_t)min(chunk0 + min(i0 + lane, chunks - 1), total - 1));
        };
        // Chunks that hold values of the row only, and all lanes have one.
        const int from = shift ? 1 : 0, to = min(chunk0 + chunks, (shift + vocab) / L::kPer);
        u32x4 c0 = load(0), c1 = load(64), c2 = load(128), c3 = load(192);
#pragma unroll 1
        for (int i0 = 0; i0 < chunks; i0 += 64) {
            u32x4 c = c0;
            c0 = c1;
            c1 = c2;
            c2 = c3;
            if (i0 + 256 < chunks) c3 = load(i0 + 256);
            const int at = (chunk0 + i0 + lane) * L::kPer - shift;
            if (chunk0 + i0 < from || chunk0 + i0 + 64 > to) {
#pragma unroll
                for (int e = 0; e < L::kPer; ++e)
                    if (i0 + lane >= chunks || (uint32_t)(at + e) >= (uint32_t)vocab) L::hide(c, e);
            }
#pragma unroll 1
            for (int e = 0; e < L::kPer; e += 4) {
#pragma unroll
                for (int j = 0; j < 4; ++j) f(L::get(c, j), at + e + j);
                if constexpr (L::kPer == 8) c = (u32x4){c[2], c[3], 0u, 0u};
            }
        }
    }
};

// A border among the bins: the first that reached it, and the counts and weights before it
// and up to it.
struct SampleBin {
    int bin, count_before, count;
    double mass_before, mass;
};

// By the last slice of a row: the others' results are read where they are coherent.
__device__ __forceinline__ SampleBorder find_border(const SampleArgs &a, const SampleRow &f, int row,
                                                    float scale, const uint64_t *own_hist,
                                                    int *s_wave_i, double *s_wave_d,
                                                    SampleBin *s_bin) {
    constexpr int kMine = kSampleBins / kSampleThreads;
    static_assert(kSamplePerOctave == 64.f, "an octave for a wave");
    // Each lane one slice: the row's maximum, and by how many bins theirs are below.
    const int lane = lane_id(), own = threadIdx.x;
    const uint64_t *head =
        (const uint64_t *)(a.slices + row * a.slices_n + min(lane, a.slices_n - 1));
    const uint64_t h0 = __hip_atomic_load(head, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const uint64_t h1 = __hip_atomic_load(head + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const float its_max = __uint_as_float((uint32_t)h0), max = wave_max(its_max);
    const int values = wave_sum_i(lane < a.slices_n ? (int)(h1 >> 32) : 0);
    const float place = sample_place(max, scale);
    const int bin = sample_top(place);
    const int by = its_max > -__builtin_inff() ? min(bin - (int)(uint32_t)h1, kSampleBins) : kSampleBins;
    // A wave has bins next to each other, an octave at a time.
    const int r0 = kMine * 64 * wave_index() + lane;
    if (own < 3) s_bin[own].bin = kSampleBins - 1;
    uint64_t sum_count[kMine] = {}, sum_mass[kMine] = {};
    // Several slices' loads on their way at once: each takes more than a microsecond.
    constexpr int kAtOnce = 3;
    if (a.slices_n == 1) {
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            const uint64_t v = own_hist[r0 + 64 * j];
            sum_count[j] = v >> 44;
            sum_mass[j] = v & ((1ull << 44) - 1);
        }
    } else {
        for (int s0 = 0; s0 < a.slices_n; s0 += kAtOnce) {
            uint64_t v[kAtOnce][kMine];
#pragma unroll
            for (int y = 0; y < kAtOnce; ++y) {
                const int sl = min(s0 + y, a.slices_n - 1), off = __builtin_amdgcn_readlane(by, sl);
                const uint64_t *hist = a.hist + ((int64_t)row * a.slices_n + sl) * kSampleBins;
#pragma unroll
                for (int j = 0; j < kMine; ++j)
                    v[y][j] = __hip_atomic_load(hist + max_i(r0 + 64 * j - off, 0),
                                                __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
#pragma unroll
            for (int y = 0; y < kAtOnce; ++y) {
                const int off =
                    s0 + y < a.slices_n ? __builtin_amdgcn_readlane(by, s0 + y) : kSampleBins;
#pragma unroll
                for (int j = 0; j < kMine; ++j) {
                    if (r0 + 64 * j < off) v[y][j] = 0;
                    sum_count[j] += v[y][j] >> 44;
                    sum_mass[j] += v[y][j] & ((1ull << 44) - 1);
                }
            }
        }
    }
    // Up to and with each bin; weights in units of the maximum's, up to a factor that
    // all share.
    double unit = 0x1p-24 * __builtin_ldexp(exp2_64(fmin(((double)(bin + 1) - (double)place - lane) *
                                                             (1.0 / kSamplePerOctave), 1.0)),
                                            -kMine * wave_index());
    int count[kMine], here = 0;
    double mass[kMine], here_mass = 0.0;
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
        // The last bin has what is left; its weights, below 2^-63 each, do not show.
        const bool is = r0 + 64 * j < kSampleBins - 1;
        int all;
        const int n = is ? (int)sum_count[j] : 0;
        count[j] = here + wave_excl_scan(n, &all) + n;
        here += all;
        mass[j] = here_mass + wave_scan_d(is ? (double)sum_mass[j] * unit : 0.0);
        here_mass = lane_d(mass[j], 63);
        unit *= 0.5;
    }
    __syncthreads();
    if (lane == 0) {
        s_wave_i[wave_index()] = here;
        s_wave_d[wave_index()] = here_mass;
    }
    __syncthreads();
    int all_count = 0, c0 = 0;
    double all_mass = 0.0, m0 = 0.0;
#pragma unroll
    for (int w = 0; w < kSampleWaves; ++w) {
        if (w == wave_index()) {
            c0 = all_count;
            m0 = all_mass;
        }
        all_count += s_wave_i[w];
        all_mass += s_wave_d[w];
    }
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
        count[j] = r0 + 64 * j < kSampleBins - 1 ? count[j] + c0 : values;
        mass[j] += m0;
    }
    // s_bin[k]: the first bin that `reached` (the last one always is).
    auto first_bin = [&](int k, auto reached) {
        int r = kSampleBins - 1;
#pragma unroll
        for (int j = kMine - 1; j >= 0; --j) {
            const uint64_t are = __ballot(reached(j));
            if (are) r = kMine * 64 * wave_index() + 64 * j + __builtin_ctzll(are);
        }
        if (lane == 0) atomicMin(&s_bin[k].bin, r);
        __syncthreads();
        r = s_bin[k].bin;
        // Its lane tells what is there, and the one before it.
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            if (r0 + 64 * j == r) {
                s_bin[k].count = count[j];
                s_bin[k].mass = mass[j];
            }
            if (r0 + 64 * j == r - 1) {
                s_bin[k].count_before = count[j];
                s_bin[k].mass_before = mass[j];
            }
            if (r == 0 && own == 0 && j == 0) {
                s_bin[k].count_before = 0;
                s_bin[k].mass_before = 0.0;
            }
        }
        __syncthreads();
        return s_bin[k];
    };
    int top = 0, bottom = kSampleBins - 1, above = 0, upto = values;
    double lo = all_mass, hi = all_mass;
    if (f.top_k) {
        const SampleBin k = first_bin(0, [&](int j) { return count[j] >= f.top_k; });
        top = bottom = k.bin;
        above = k.count_before;
        upto = k.count;
        lo = k.mass_before;
        hi = k.mass;
    }
    // (Where all are in the last bin, nothing is known of their weights.)
    if (f.by_p && all_count == 0) {
        top = 0;
        above = 0;
    } else if (f.by_p) {
        // What the sums of weights may be off by: 2^-23 each for the power and for the
        // 24 bits, and for places and their scale, rounded to 24 bits both (ln 2 / 64 a
        // place; more, where they are off by many).
        const double off = 0x1p-20 + (fabs((double)place) + kSampleBins) * 0x1p-24 * 0.035;
        const double least = f.top_p * lo * (1.0 - off), most = f.top_p * hi * (1.0 + off);
        const SampleBin p =
            first_bin(1, [&](int j) { return mass[j] * (1.0 + off) >= least; });
        if (!f.top_k || p.bin < top) {
            top = p.bin;
            above = p.count_before;
        }
        if (!f.top_k) {
            const SampleBin q =
                first_bin(2, [&](int j) { return mass[j] * (1.0 - off) >= most; });
            bottom = q.bin;
            upto = q.count;
        }
    }
    // The smallest values in bins above `top`, and in `bottom`: of the keys from +inf's to
    // that of the lowest finite value the last for which that holds, 64 tried at once.
    auto last_key = [&](int below) {
        uint32_t lo = sample_key(__builtin_inff()), hi = sample_key(-3.402823466e38f);
        while (lo < hi) {
            const uint32_t step = ((hi - lo) >> 6) + 1, key = lo + min(step * lane, hi - lo);
            const int r = bin - sample_bin(sample_place(sample_value(key), scale));
            const int n = __builtin_popcountll(__ballot(min(r, kSampleBins - 1) < below));
            if (n == 0) return ~0u;
            lo += min(step * (n - 1), hi - lo);
            hi = min(hi, lo + step - 1);
        }
        return lo;
    };
    SampleBorder b;
    const uint32_t key = last_key(top), low_key = last_key(bottom + 1);
    b.top = key == ~0u ? __builtin_nanf("") : sample_value(key);
    b.bottom = sample_value(low_key);
    b.above = above;
    b.listed = upto - above;
    return b;
}

template <int Type>
__global__ __launch_bounds__(kSampleThreads, 4) void k_sample_scan(const SampleArgs a) {
    __shared__ uint64_t s_hist[kSampleBins];
    __shared__ double s_wave_d[kSampleWaves];
    __shared__ int s_wave_i[kSampleWaves];
    __shared__ SampleBin s_bin[3];
    __shared__ uint32_t s_last;
    __shared__ float s_max[kSampleWaves];
    __shared__ int s_first[kSampleWaves], s_count[kSampleWaves];
    const int row = (int)blockIdx.x / a.slices_n, slice = (int)blockIdx.x % a.slices_n;
    const int lane = lane_id(), wave = wave_index();
    const SampleRow f = sample_row(a, row);
    Segment<Type> seg(a, row, slice * kSampleWaves + wave, a.chunks);
    const bool binned = !f.greedy && (f.top_k || f.by_p);
    if (binned)
        for (int i = threadIdx.x; i < kSampleBins; i += kSampleThreads) s_hist[i] = 0;
    float max = -__builtin_inff();
    seg.each(a.vocab, [&](float x, int) { max = fmaxf(max, x); });
    max = wave_max(max);
    int first = 0x7FFFFFFF;
    if (f.greedy) {
        seg.each(a.vocab, [&](float x, int i) { first = x == max ? min(first, i) : first; });
        first = wave_min_i(first);
    }
    if (lane == 0) {
        s_max[wave] = max;
        s_first[wave] = first;
    }
    __syncthreads();
    max = s_max[0];
#pragma unroll
    for (int w = 1; w < kSampleWaves; ++w) max = fmaxf(max, s_max[w]);
    first = 0x7FFFFFFF;
#pragma unroll
    for (int w = 0; w < kSampleWaves; ++w) first = s_max[w] == max ? min(first, s_first[w]) : first;
    const float scale = sample_scale(f.temperature);
    const int top = sample_top(sample_place(max, scale));
    uint64_t *mine = (uint64_t *)(a.slices + blockIdx.x);
    if (threadIdx.x == 0)
        __hip_atomic_store(mine, (uint64_t)(uint32_t)first << 32 | __float_as_uint(max),
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (!binned) return;
    int low = 0;
    if (max > -__builtin_inff())
        seg.each(a.vocab, [&](float x, int) {
            const float place = sample_place(x, scale);
            const int r = top - sample_bin(place);
            // 2^24 times the weight in units of that of the bin's upper end
            const float w = exp2_(fmaf(__builtin_amdgcn_fractf(place), 1.f / kSamplePerOctave,
                                       24.f - 1.f / kSamplePerOctave));
            if (r < kSampleBins - 1)
                __hip_atomic_fetch_add(&s_hist[r], 1ull << 44 | (uint32_t)w, __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_WORKGROUP);
            else
                low += x > -__builtin_inff();
        });
    __syncthreads();
    // All of its values: those that are not in the last bin of this slice may be in the
    // row's.
    int count = low;
    uint64_t *hist = a.hist + (int64_t)blockIdx.x * kSampleBins;
#pragma unroll
    for (int j = 0; j < kSampleBins / kSampleThreads; ++j) {
        const int i = threadIdx.x + kSampleThreads * j;
        const uint64_t v = s_hist[i];
        count += (int)(v >> 44);
        if (a.slices_n > 1)
            __hip_atomic_store(hist + i, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    count = wave_sum_i(count);
    if (lane == 0) s_count[wave] = count;
    __syncthreads();
    if (threadIdx.x == 0) {
        count = 0;
#pragma unroll
        for (int w = 0; w < kSampleWaves; ++w) count += s_count[w];
        __hip_atomic_store(mine + 1, (uint64_t)(uint32_t)count << 32 | (uint32_t)top,
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    wait_vm_all();
    __syncthreads();
    if (threadIdx.x == 0)
        s_last = __hip_atomic_fetch_add(a.counters + row, 1u, __ATOMIC_RELAXED,
                                        __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (s_last != (uint32_t)a.slices_n - 1) return;
    const SampleBorder b = find_border(a, f, row, scale, s_hist, s_wave_i, s_wave_d, s_bin);
    if (threadIdx.x == 0) {
        a.borders[row] = b;
        store_agent(a.counters + row, 0u);
    }
}

// Sorts n different 64-bit keys in LDS, K a thread: in registers among a thread's own, by
// lane exchanges within a wave, and through LDS between waves only (a stage through LDS
// takes 0.2 us, most of it the barriers).
template <int K>
__device__ __forceinline__ void sort_keys(uint64_t *s, int n) {
    const int own = threadIdx.x;
    uint64_t v[K];
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = K * own + k < n ? s[K * own + k] : ~0ull;
    int n2 = K;
    while (n2 < n) n2 <<= 1;
#pragma unroll 1
    for (int size = 2; size <= n2; size <<= 1)
#pragma unroll 1
        for (int by = size >> 1; by > 0; by >>= 1) {
            if (by < K) {
#pragma unroll
                for (int b = 1; b < K; b <<= 1) {
                    if (b != by) continue;
#pragma unroll
                    for (int k = 0; k < K; ++k) {
                        if (k & b) continue;
                        const bool up = ((K * own + k) & size) == 0;
                        const uint64_t x = v[k], y = v[k | b];
                        const bool swap = (x > y) == up;
                        v[k] = swap ? y : x;
                        v[k | b] = swap ? x : y;
                    }
                }
                continue;
            }
            const int lanes = by / K;
            const bool keep_min = ((K * own & by) == 0) == ((K * own & size) == 0);
            if (lanes >= 64) {
                __syncthreads();
#pragma unroll
                for (int k = 0; k < K; ++k) s[kSampleThreads * k + own] = v[k];
                __syncthreads();
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                uint64_t o;
                if (lanes >= 64) {
                    o = s[kSampleThreads * k + (own ^ lanes)];
                } else {
                    const uint32_t lo = __shfl_xor((uint32_t)v[k], lanes);
                    o = (uint64_t)(uint32_t)__shfl_xor((uint32_t)(v[k] >> 32), lanes) << 32 | lo;
                }
                v[k] = (o < v[k]) == keep_min ? o : v[k];
            }
        }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (K * own + k < n) s[K * own + k] = v[k];
    __syncthreads();
}

template <int Type>
struct SampleLds {
    union {
        uint64_t list[kSampleList];
        struct {
            uint32_t count[kSampleKeyBins];
            unsigned long long mass[kSampleKeyBins];
        } bins;
    };
    union {
        double wave_d[kSampleWaves];
        uint64_t wave_u[kSampleWaves];
    };
    int wave_i[kSampleWaves];
    double seg[kSampleSegments + 1];
    union {
        double upto[kSampleSegments];          // of a segment's kept ones at the border
        unsigned long long quanta[kSampleSegments];
        int equal[kSampleSegments];            // values like the border's in a segment
    };
    int n, found;
    uint32_t last;
    int token, count, before, bin;
    uint64_t mass_before;
};
// Of k_sample_plain.
struct SamplePlainLds {
    double wave_d[kSampleWaves];
    double seg[kSampleSegments + 1];
    int found;
    uint32_t last;
};

// The first of n places that `holds`; where none does, the last that `some`, or 0.
template <class Lds, class Holds, class Some>
__device__ __forceinline__ int first_place(Lds &s, int n, Holds holds, Some some) {
    __syncthreads();
    if (threadIdx.x == 0) s.found = 0x7FFFFFFF;
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += kSampleThreads)
        if (holds(j)) {
            atomicMin(&s.found, j);
            break;
        }
    __syncthreads();
    int who = s.found;
    if (who != 0x7FFFFFFF) return who;
    __syncthreads();
    if (threadIdx.x == 0) s.found = 0;
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += kSampleThreads)
        if (some(j)) atomicMax(&s.found, j);
    __syncthreads();
    return s.found;
}

// The token of a row whose sums up to each segment are in s.seg: the segment, then the
// place in it.  A thread takes a few chunks next to each other.  weight(x), and
// is_kept(x, index).
template <int Type, class Lds, class Weight, class Is>
__device__ __forceinline__ void draw_token(const SampleArgs &a, int row, const SampleRow &f,
                                           Lds &s, Weight weight, Is is_kept) {
    typedef Logits<Type> L;
    const int own = threadIdx.x, segments = a.draws * kSampleWaves;
    const double total = s.seg[segments], target = (double)f.u * total;
    const int who = first_place(
        s, segments, [&](int j) { return s.seg[j + 1] > target && s.seg[j + 1] > s.seg[j]; },
        [&](int j) { return s.seg[j + 1] > s.seg[j]; });
    const Segment<Type> seg(a, row, who, a.draw_chunks);
    const int per = (a.draw_chunks + kSampleThreads - 1) / kSampleThreads, first = own * per;
    auto each_kept = [&](auto take) {
#pragma unroll 1
        for (int j = 0; j < per; ++j) {
            const int in = first + j, at = (seg.chunk0 + in) * L::kPer - seg.shift;
            u32x4 c = ld16(seg.row - seg.shift * L::kBytes +
                           16 * (int64_t)min(seg.chunk0 + in, seg.total - 1));
#pragma unroll 1
            for (int e = 0; e < L::kPer; e += 4) {
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float x = L::get(c, y);
                    const int i = at + e + y;
                    const bool is = in < a.draw_chunks && (uint32_t)i < (uint32_t)a.vocab &&
                                    x > -__builtin_inff() && is_kept(x, i);
                    take(i, is ? weight(x) : 0.0);
                }
                if constexpr (L::kPer == 8) c = (u32x4){c[2], c[3], 0u, 0u};
            }
        }
    };
    double sum = 0.0, all;
    each_kept([&](int, double w) { sum += w; });
    const double before = s.seg[who] + block_scan_d(sum, &all, s.wave_d);
    // (Where rounding leaves nobody beyond the target, the last that is kept.)
    const int by = first_place(s, kSampleThreads, [&](int) { return sum > 0.0 && before + sum > target; },
                               [&](int) { return sum > 0.0; });
    if (own == by) {
        double at = before, of = 1.0;
        int token = 0;
        bool found = false;
        each_kept([&](int i, double w) {
            at += w;
            if (!found && w > 0.0) {
                token = i;
                of = w;
                found = at > target;
            }
        });
        a.token[row] = token;
        a.logprob[row] = (float)log(of / total);
    }
}

// All segments of a row, by one workgroup: f(segment, its index).
template <int Type, class F>
__device__ __forceinline__ void each_segment(const SampleArgs &a, int row, F f) {
    for (int i = wave_index(); i < a.draws * kSampleWaves; i += kSampleWaves) {
        Segment<Type> seg(a, row, i, a.draw_chunks);
        f(seg, i);
    }
}

// Of the listed values with keys from lo to hi: the key at which a sum reaches `target`,
// by count or by weight (in 2^-44), with what is before it in s.before and s.mass_before
// (if weights are summed) and how often it is there in s.count.  base: the sum before the
// first of them.
template <int Type, class Listed, class Weight>
__device__ __forceinline__ uint32_t border_key(const SampleArgs &a, int row, SampleLds<Type> &s,
                                               bool by_mass, bool summed, double base,
                                               double target, uint32_t lo, uint32_t hi,
                                               Listed listed, Weight weight_of) {
    int before = 0;
    uint64_t mass_before = 0;
    for (;;) {
        int shift = 0;
        while ((hi - lo) >> shift >= kSampleKeyBins) ++shift;
        __syncthreads();
        for (int i = threadIdx.x; i < kSampleKeyBins; i += kSampleThreads) {
            s.bins.count[i] = 0;
            s.bins.mass[i] = 0;
        }
        __syncthreads();
        each_segment<Type>(a, row, [&](const Segment<Type> &seg, int) {
            seg.each(a.vocab, [&](float x, int) {
                const uint32_t key = sample_key(x);
                const bool in = listed(x) && key >= lo && key <= hi;
                const uint64_t here = __ballot(in);
                if (!here) return;
                const uint64_t m = summed ? (uint64_t)(weight_of(x) * 0x1p44) : 0;
                // (All of one value, as equal logits are: one addition for the wave.)
                const int first = __builtin_ctzll(here);
                const uint32_t value = __builtin_amdgcn_readlane(key, first);
                const bool one = __ballot(in && key == value) == here;
                const int n = one ? __builtin_popcountll(here) : 1;
                if (one ? lane_id() == first : in) {
                    atomicAdd(&s.bins.count[(key - lo) >> shift], (uint32_t)n);
                    if (summed) atomicAdd(&s.bins.mass[(key - lo) >> shift], (unsigned long long)m * n);
                }
            });
        });
        __syncthreads();
        // The bin at which the sum reaches the target, or the last that holds any.
        constexpr int kMine = kSampleKeyBins / kSampleThreads;
        const int r0 = kMine * (int)threadIdx.x;
        int here = 0, all_count;
        uint64_t here_mass = 0, all_mass;
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            here += (int)s.bins.count[r0 + j];
            here_mass += s.bins.mass[r0 + j];
        }
        const int c0 = before + block_scan_i(here, &all_count, s.wave_i);
        const uint64_t m0 = mass_before + block_scan_d(here_mass, &all_mass, s.wave_u);
        auto reached = [&](int c, uint64_t m) {
            return by_mass ? base + (double)m * 0x1p-44 >= target : base + (double)c >= target;
        };
        const int who = first_place(
            s, kSampleThreads, [&](int) { return here && reached(c0 + here, m0 + here_mass); },
            [&](int) { return here != 0; });
        if ((int)threadIdx.x == who) {
            int c = c0;
            uint64_t m = m0;
            for (int j = 0; j < kMine; ++j) {
                const int n = (int)s.bins.count[r0 + j];
                if (!n) continue;
                s.bin = r0 + j;
                s.count = n;
                s.before = c;
                s.mass_before = m;
                c += n;
                m += s.bins.mass[r0 + j];
                if (reached(c, m)) break;
            }
        }
        __syncthreads();
        before = s.before;
        mass_before = s.mass_before;
        lo += (uint32_t)s.bin << shift;
        hi = min(hi, lo + ((1u << shift) - 1));
        if (shift == 0 || lo == hi) return lo;
    }
}

template <int Type>
__global__ __launch_bounds__(kSampleThreads, 4) void k_sample_draw(const SampleArgs a) {
    typedef Logits<Type> L;
    __shared__ SampleLds<Type> s;
    const int row = (int)blockIdx.x / a.draws, slice = (int)blockIdx.x % a.draws;
    const int lane = lane_id(), wave = wave_index();
    const Segment<Type> seg(a, row, slice * kSampleWaves + wave, a.draw_chunks);
    const SampleRow f = sample_row(a, row);
    SampleBorder b = a.borders[row];
    const SampleSlice its = a.slices[row * a.slices_n + min(lane, a.slices_n - 1)];
    const float max = wave_max(its.max);
    if (max == -__builtin_inff() || f.greedy) {
        if (slice == 0 && wave == 0) {
            const int first = wave_min_i(its.max == max ? its.first : 0x7FFFFFFF);
            if (lane == 0) {
                a.token[row] = max == -__builtin_inff() ? -1 : first;
                a.logprob[row] = max == -__builtin_inff() ? max : 0.f;
            }
        }
        return;
    }
    const double c = 1.44269504088896340736 / (double)f.temperature, min_p = f.min_p;
    if (!f.top_k && !f.by_p) b = {-3.402823466e38f, -3.402823466e38f, a.vocab, 0};   // all are above
    auto weight_of = [&](float x) { return sample_weight(x, max, c); };
    auto kept_weight = [&](float x) {
        const double w = weight_of(x);
        return w >= min_p ? w : 0.0;
    };
    auto is_listed = [&](float x) { return x >= b.bottom && !(x >= b.top); };
    const bool wide = b.listed > kSampleList;
    const bool rest = f.by_p && !f.top_k;     // the sum of all weights is needed
    uint32_t *arrived = a.counters + row;
    uint64_t *list = a.list + (int64_t)blockIdx.x * kSampleList;
    if (threadIdx.x == 0) s.n = 0;
    __syncthreads();
    double above = 0.0, kept = 0.0, total = 0.0;
    uint32_t key_lo = ~0u, key_hi = 0;
    auto list_it = [&](float x, int i) {
        const uint32_t key = sample_key(x);
        if (wide) {
            key_lo = min(key_lo, key);
            key_hi = max_u(key_hi, key);
        } else {
            const int at = atomicAdd(&s.n, 1);
            if (at < kSampleList)
                __hip_atomic_store(list + at, (uint64_t)key << 32 | (uint32_t)i, __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
        }
    };
    if (rest)
        seg.each(a.vocab, [&](float x, int i) {
            const double w = weight_of(x);
            total += w;
            const double is = x >= b.top ? w : 0.0;
            above += is;
            if (min_p > 0.0) kept += is >= min_p ? is : 0.0;
            if (is_listed(x)) list_it(x, i);
        });
    else
        seg.each(a.vocab, [&](float x, int i) {
            if (x >= b.top) {
                const double w = weight_of(x);
                above += w;
                if (min_p > 0.0) kept += w >= min_p ? w : 0.0;
            } else if (x >= b.bottom) {
                list_it(x, i);
            }
        });
    above = wave_sum_d(above);
    kept = min_p > 0.0 ? wave_sum_d(kept) : above;
    if (rest) total = wave_sum_d(total);
    if (wide)
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1) {
            key_lo = min(key_lo, (uint32_t)__shfl_xor((int)key_lo, m));
            key_hi = max_u(key_hi, (uint32_t)__shfl_xor((int)key_hi, m));
        }
    if (lane == 0) {
        const int64_t at = (int64_t)blockIdx.x * kSampleWaves + wave;
        double *to = a.sums + at * kSampleSlots;
        store_agent_d(to, above);
        store_agent_d(to + 1, kept);
        store_agent_d(to + 2, total);
        if (wide)
            __hip_atomic_store(a.keys + at, (uint64_t)key_hi << 32 | key_lo, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (threadIdx.x == 0)
        __hip_atomic_store(a.listed + blockIdx.x, min(s.n, kSampleList), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
    wait_vm_all();
    __syncthreads();
    if (threadIdx.x == 0)
        s.last = __hip_atomic_fetch_add(arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (s.last != (uint32_t)a.draws - 1) return;

    // The last workgroup of the row.
    if (threadIdx.x == 0) store_agent(arrived, 0u);
    const int listed = load_agent(a.listed + row * a.draws + min(lane, a.draws - 1));
    const int segments = a.draws * kSampleWaves;
    const double *sums = a.sums + (int64_t)row * segments * kSampleSlots;
    above = kept = total = 0.0;
    if ((int)threadIdx.x < segments) {
        above = load_agent_d(sums + threadIdx.x * kSampleSlots);
        kept = load_agent_d(sums + threadIdx.x * kSampleSlots + 1);
        total = load_agent_d(sums + threadIdx.x * kSampleSlots + 2);
    }
    double all_above = 0.0, all_weights = 0.0, all_kept;
    const double kept_before = block_scan_d(kept, &all_kept, s.wave_d);
    if (f.by_p) block_scan_d(above, &all_above, s.wave_d);
    if (rest) block_scan_d(total, &all_weights, s.wave_d);

    // The border: values up to this one, by key and index, are kept, and those above.
    uint64_t border = 0;
    bool some = false;          // any of the listed ones are
    const int per_segment = a.draw_chunks * L::kPer;
    const int own = (int)threadIdx.x;
    if (b.listed && !wide) {
        // All slices' shares of the list: the n-th of all is the share's whose first is the
        // last one up to n.
        int n;
        const int first = wave_excl_scan(lane < a.draws ? listed : 0, &n);
        for (int j0 = 64 * wave; j0 < n; j0 += kSampleThreads) {
            const int j = j0 + lane;
            int share = 0;
            for (int i = 1; i < a.draws; ++i) {
                const int at = __builtin_amdgcn_readlane(first, i);
                share = j >= at ? i : share;
            }
            const int at = __shfl(first, share);
            if (j < n)
                s.list[j] = __hip_atomic_load(
                    a.list + ((int64_t)row * a.draws + share) * kSampleList + j - at,
                    __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        for (int i = own; i < segments; i += kSampleThreads) s.quanta[i] = 0;
        __syncthreads();
        if (n <= kSampleThreads) sort_keys<1>(s.list, n);
        else if (n <= 2 * kSampleThreads) sort_keys<2>(s.list, n);
        else sort_keys<8>(s.list, n);
        int take = f.top_k ? min(n, f.top_k - b.above) : n;
        if (f.by_p) {
            const int per = (n + kSampleThreads - 1) / kSampleThreads, j0 = own * per;
            auto weight_at = [&](int j) { return weight_of(sample_value((uint32_t)(s.list[j] >> 32))); };
            double sum = 0.0, all;
            for (int j = j0; j < min(j0 + per, take); ++j) sum += weight_at(j);
            double before = all_above + block_scan_d(sum, &all, s.wave_d);
            const double target = (double)f.top_p * (rest ? all_weights : all_above + all);
            int count = 0, in;
            for (int j = j0; j < min(j0 + per, take); ++j) {
                count += before < target;
                before += weight_at(j);
            }
            block_scan_i(count, &in, s.wave_i);
            take = max_i(in, b.above ? 0 : 1);
        }
        some = take > 0;
        border = some ? s.list[take - 1] : 0;
        // What is kept of it, by segment: as integers, whose sums have no order.
        for (int j = own; j < take; j += kSampleThreads) {
            const double w = kept_weight(sample_value((uint32_t)(s.list[j] >> 32)));
            const int at = (int)(uint32_t)s.list[j] + seg.shift;
            atomicAdd(&s.quanta[at / (a.draw_chunks * L::kPer)],
                      (unsigned long long)__builtin_rint(w * 0x1p44));
        }
        __syncthreads();
        const double mine = own < segments ? (double)s.quanta[own] * 0x1p-44 : 0.0;
        double all;
        const double before = block_scan_d(mine, &all, s.wave_d);
        if (own <= segments)
            s.seg[own] = own < segments ? kept_before + before : all_kept + all;
        __syncthreads();
    } else if (wide) {
        uint32_t lo = ~0u, hi = 0;
        for (int i = 0; i < segments; ++i) {
            const uint64_t k = __hip_atomic_load(a.keys + (int64_t)row * segments + i,
                                                 __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            lo = min(lo, (uint32_t)k);
            hi = max_u(hi, (uint32_t)(k >> 32));
        }
        auto quantum = [&](uint32_t key) { return (uint64_t)(weight_of(sample_value(key)) * 0x1p44); };
        uint32_t key = hi;
        int equal = 0x7FFFFFFF, count = 0;      // kept of those with this key, and all
        double mass = all_weights;
        if (f.top_k) {
            key = border_key<Type>(a, row, s, false, f.by_p, b.above, f.top_k, lo, hi, is_listed,
                                   weight_of);
            count = s.count;
            equal = min(count, f.top_k - b.above - s.before);
            mass = all_above + (double)(s.mass_before + equal * quantum(key)) * 0x1p-44;
        }
        if (f.by_p) {
            const double target = (double)f.top_p * mass;
            const uint32_t its = border_key<Type>(a, row, s, true, true, all_above, target, lo, key,
                                                  is_listed, weight_of);
            const double w = (double)quantum(its) * 0x1p-44;
            const double left = target - (all_above + (double)s.mass_before * 0x1p-44);
            const double more = w > 0.0 ? __builtin_ceil(left / w) : 0x1p31;
            count = s.count;
            const int n = (int)fmin(fmax(more, 1.0), (double)count);
            equal = its == key ? min(equal, n) : n;
            key = its;
        }
        some = equal > 0;
        border = (uint64_t)key << 32 | 0xFFFFFFFFu;
        __syncthreads();
        if (equal < count) {
            // Equal ones are kept by index: the index of the last that is.
            each_segment<Type>(a, row, [&](const Segment<Type> &seg, int i) {
                int n = 0;
                seg.each(a.vocab, [&](float x, int) { n += x > -__builtin_inff() && sample_key(x) == key; });
                n = wave_sum_i(n);
                if (lane == 0) s.equal[i] = n;
            });
            __syncthreads();
            int at = 0, before = 0;
            while (before + s.equal[at] < equal) before += s.equal[at++];
            if (wave == 0) {
                Segment<Type> seg(a, row, at, a.draw_chunks);
                        int from = at * per_segment - seg.shift - 1, to = from + per_segment;
                while (to - from > 1) {       // (as many as are needed are up to `to`)
                    const int mid = (from + to) >> 1;
                    int n = 0;
                    seg.each(a.vocab, [&](float x, int i) {
                        n += x > -__builtin_inff() && sample_key(x) == key && i <= mid;
                    });
                    if (wave_sum_i(n) >= equal - before) to = mid;
                    else from = mid;
                }
                if (lane == 0) s.token = to;
            }
            __syncthreads();
            border = (uint64_t)key << 32 | (uint32_t)s.token;
            __syncthreads();
        }
        each_segment<Type>(a, row, [&](const Segment<Type> &seg, int i) {
            double sum = 0.0;
            seg.each(a.vocab, [&](float x, int at) {
                const bool is = some && is_listed(x) &&
                                ((uint64_t)sample_key(x) << 32 | (uint32_t)at) <= border;
                if (is) sum += kept_weight(x);
            });
            sum = wave_sum_d(sum);
            if (lane == 0) s.upto[i] = sum;
        });
        __syncthreads();
        double all;
        const double before = block_scan_d(own < segments ? s.upto[own] : 0.0, &all, s.wave_d);
        if (own <= segments)
            s.seg[own] = own < segments ? kept_before + before : all_kept + all;
        __syncthreads();
    } else {
        if (own <= segments) s.seg[own] = own < segments ? kept_before : all_kept;
        __syncthreads();
    }

    draw_token<Type>(a, row, f, s, kept_weight, [&](float x, int i) {
        return x >= b.top ||
               (some && ((uint64_t)sample_key(x) << 32 | (uint32_t)i) <= border);
    });
}

// Rows without filters.
template <int Type>
__global__ __launch_bounds__(kSampleThreads, 4) void k_sample_plain(const SampleArgs a) {
    __shared__ SamplePlainLds s;
    const int row = (int)blockIdx.x / a.draws, slice = (int)blockIdx.x % a.draws;
    const int lane = lane_id(), wave = wave_index(), own = threadIdx.x;
    const SampleRow f = sample_row(a, row);
    const double c = 1.44269504088896340736 / (double)f.temperature;
    // The segment's maximum, where it is first, and the weights in units of its own.
    {
        const Segment<Type> seg(a, row, slice * kSampleWaves + wave, a.draw_chunks);
        float max = -__builtin_inff();
        seg.each(a.vocab, [&](float x, int) { max = fmaxf(max, x); });
        max = wave_max(max);
        double sum = 0.0;
        int first = 0x7FFFFFFF;
        if (f.greedy) {
            seg.each(a.vocab, [&](float x, int i) { first = x == max ? min(first, i) : first; });
            first = wave_min_i(first);
        } else if (max > -__builtin_inff()) {
            seg.each(a.vocab, [&](float x, int) {
                if (x > -__builtin_inff()) sum += sample_weight(x, max, c);
            });
            sum = wave_sum_d(sum);
        }
        if (lane == 0) {
            double *to = a.sums + ((int64_t)blockIdx.x * kSampleWaves + wave) * kSampleSlots;
            store_agent_d(to, sum);
            __hip_atomic_store((uint64_t *)to + 1, (uint64_t)(uint32_t)first << 32 | __float_as_uint(max),
                               __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    wait_vm_all();
    __syncthreads();
    uint32_t *arrived = a.counters + row;
    if (own == 0)
        s.last = __hip_atomic_fetch_add(arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (s.last != (uint32_t)a.draws - 1) return;
    if (own == 0) store_agent(arrived, 0u);
    const int segments = a.draws * kSampleWaves;
    // All waves the same: a few segments a lane.
    constexpr int kEach = kSampleSegments / 64;
    const double *sums = a.sums + (int64_t)row * segments * kSampleSlots;
    double part[kEach];
    float its[kEach], max = -__builtin_inff();
    int first[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int i = min(64 * j + lane, segments - 1);
        part[j] = load_agent_d(sums + i * kSampleSlots);
        const uint64_t m = __hip_atomic_load((const uint64_t *)(sums + i * kSampleSlots) + 1,
                                             __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        its[j] = __uint_as_float((uint32_t)m);
        first[j] = (int)(m >> 32);
        max = fmaxf(max, its[j]);
    }
    max = wave_max(max);
    if (max == -__builtin_inff() || f.greedy) {
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int j = 0; j < kEach; ++j) at = its[j] == max ? min(at, first[j]) : at;
        at = wave_min_i(at);
        if (own == 0) {
            a.token[row] = max == -__builtin_inff() ? -1 : at;
            a.logprob[row] = max == -__builtin_inff() ? max : 0.f;
        }
        return;
    }
    double before = 0.0;
#pragma unroll 1
    for (int j = 0; j < kEach && 64 * j < segments; ++j) {
        const int i = 64 * j + lane;
        const bool is = i < segments && its[j] > -__builtin_inff();
        const double inc = before + wave_scan_d(is ? part[j] * sample_weight(its[j], max, c) : 0.0);
        if (wave == 0 && i < segments) s.seg[i + 1] = inc;
        before = lane_d(inc, 63);
    }
    if (own == 0) s.seg[0] = 0.0;
    __syncthreads();
    draw_token<Type>(a, row, f, s, [&](float x) { return sample_weight(x, max, c); },
                     [](float, int) { return true; });
}

}  // namespace serve
}  // namespace moe
