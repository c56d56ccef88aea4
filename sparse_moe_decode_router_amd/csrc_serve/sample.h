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
//                   the values in them.  The last slice of a row to finish narrows
//                   the list down, by histograms of 11 bits of (value, index) a pass,
//                   to the last token that is kept; finds the segment (a wave's share
//                   of a slice) that holds the drawn one; and that.
// Bins are monotonic in the value and their counts exact, so that the list holds the
// border whatever the weights' 20 bits missed (the margin of the search covers
// that).  Where the list would be too long (thousands of equal logits at the border, or a
// top_p within 2e-5 of 1, whose border is among nearly all tokens), the passes go over the
// row instead, by one workgroup: for one row of 163840 282 us instead of 21.
//   k_sample_plain  rows without filters: each segment's maximum and sum, and the last
//                   slice draws.  One launch.
//
// What bounds it: few rows are a chain of latencies, each phase a barrier and a read of
// what other slices left (one row of 163840, bf16: 19 us a launch, most of it after the
// slices' passes of 2 and 4 us); many rows are bound by the vector unit, the 64-bit
// exponentials above all (512 rows of 100003, top-p: 53 us to scan and 98 to draw, where
// reading the logits takes 20).  Eight rows of 32003 without filters take 10 us, 64 of 163840
// 25.  No registers are spilled but one, of the draw from f32.
//   Histograms of 64-bit integers in LDS, because the order of additions must not change
//   a sum, and because the borders then come from one pass instead of one a digit.
//   More slices shorten the passes and lengthen what their last one reads: nine at most
//   for histograms of 32 KB, 32 for the sums.
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
constexpr int kSampleKeyBins = 2048;    // of a pass over the list
constexpr int kSampleIndexBits = 19;
constexpr int kSampleSlots = 3;         // sums of a segment: above, above and kept, all

struct SampleSlice {
    float max;         // -inf: nothing to draw
    int32_t first;     // index of the first value that is the maximum
    int32_t bin;       // of the maximum
    int32_t pad;       // (read as two integers of 64 bits)
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
    uint64_t *hist;           // [rows][slices][kSampleBins]: count << 44 | weights (of one: none)
    SampleBorder *borders;    // [rows]
    double *sums;             // [rows][draws][waves][kSampleSlots] (plain: the sum, the maximum)
    uint64_t *list;           // [rows][draws][kSampleList] (of one: none)
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
__device__ __forceinline__ uint64_t min_u64(uint64_t a, uint64_t b) { return a < b ? a : b; }
__device__ __forceinline__ uint64_t max_u64(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t xor_u64(uint64_t v, int lanes) {
    const uint32_t lo = __shfl_xor((uint32_t)v, lanes);
    return (uint64_t)(uint32_t)__shfl_xor((uint32_t)(v >> 32), lanes) << 32 | lo;
}

// The logits of a 16-byte chunk.
template <int Type>
struct Logits {
    static constexpr int kPer = Type == kSampleF32 ? 4 : 8;
    static constexpr int kBytes = 16 / kPer;
    static constexpr int kDrop = Type == kSampleF32 ? 0 : Type == 0 ? 16 : 13;   // bits of f32 that say nothing
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

// 2^y for y <= 0 (above: 1, NaN: 0), to 2^-44: with r = y less the nearest integer, 1 + r q(r),
// where q has the values of (2^r - 1) / r at nine Chebyshev nodes of [-1/2, 1/2].
__device__ __forceinline__ double exp2_64(double y) {
    y = fmin(fmax(y, -1100.0), 0.0);
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
// The weight of a row's values: the maximum has 1, also where it is infinite (then all
// finite ones have none); -inf and NaN have none.
struct SampleWeight {
    double max, c;      // c: log2(e) / T
    __device__ __forceinline__ SampleWeight(float of_max, float temperature) {
        const bool inf = of_max == __builtin_inff();
        max = inf ? 0x1p128 : (double)of_max;
        c = inf ? 0x1p900 : 1.44269504088896340736 / (double)temperature;
    }
    // Of the power of 2 that is the weight.
    __device__ __forceinline__ double exponent(float x) const {
        return fmin(fmax(((double)x - max) * c, -1100.0), 0.0);
    }
    __device__ __forceinline__ double operator()(float x) const {
        return exp2_64(((double)x - max) * c);
    }
};

// Order of values as unsigned integers: larger x, smaller key.  NaN counts as -inf, and
// the two zeros are equal.
__device__ __forceinline__ uint32_t sample_key(float x) {
    const uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);
    return b >> 31 ? b : ~b & 0x7FFFFFFFu;
}
__device__ __forceinline__ float sample_value(uint32_t key) {
    return __uint_as_float(key >> 31 ? key : ~key & 0x7FFFFFFFu);
}
// The order of tokens: by value, then by index.
template <int Type>
__device__ __forceinline__ uint64_t sample_order(float x, int index) {
    return (uint64_t)(sample_key(x) >> Logits<Type>::kDrop) << kSampleIndexBits | (uint32_t)index;
}
template <int Type>
__device__ __forceinline__ float sample_ordered(uint64_t order) {
    constexpr int kDrop = Logits<Type>::kDrop;
    const uint32_t key = (uint32_t)(order >> kSampleIndexBits) << kDrop;
    return sample_value(key >> 31 ? key : key | ((1u << kDrop) - 1));   // (what is dropped is zero in x)
}
__device__ __forceinline__ int sample_index(uint64_t order) {
    return (int)(order & ((1u << kSampleIndexBits) - 1));
}
// The natural logarithm of x >= 1, to 2^-40: a 32-bit one, corrected by what is left.
__device__ __forceinline__ double log_64(double x) {
    int e = __builtin_amdgcn_frexp_exp(x);
    const double y = (double)e + (double)log2_((float)__builtin_ldexp(x, -e));
    const double half = exp2_64(-0.5 * y), r = x * half * half - 1.0;   // (2^-y may be too small)
    return y * 0.69314718055994530942 + (r - 0.5 * r * r);
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
// The same of 32 bits.
template <int C, int Rows>
__device__ __forceinline__ int add_dpp_i(int v) {
    return v + __builtin_amdgcn_update_dpp(0, v, C, Rows, 0xF, false);
}
__device__ __forceinline__ int wave_scan_i(int v) {
    v = add_dpp_i<0x111, 0xF>(v);
    v = add_dpp_i<0x112, 0xF>(v);
    v = add_dpp_i<0x114, 0xF>(v);
    v = add_dpp_i<0x118, 0xF>(v);
    v = add_dpp_i<0x142, 0xA>(v);
    return add_dpp_i<0x143, 0xC>(v);
}
// Scans of K values side by side: each step waits for the one before it.
template <int C, int Rows, int K>
__device__ __forceinline__ void add_dpp_all(int *n, double *v) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
        n[k] = add_dpp_i<C, Rows>(n[k]);
        v[k] = add_dpp<C, Rows>(v[k]);
    }
}
template <int K>
__device__ __forceinline__ void wave_scan_all(int *n, double *v) {
    add_dpp_all<0x111, 0xF, K>(n, v);
    add_dpp_all<0x112, 0xF, K>(n, v);
    add_dpp_all<0x114, 0xF, K>(n, v);
    add_dpp_all<0x118, 0xF, K>(n, v);
    add_dpp_all<0x142, 0xA, K>(n, v);
    add_dpp_all<0x143, 0xC, K>(n, v);
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
    const int inc = wave_scan_i(v);
    __syncthreads();
    if (lane_id() == 63) s_wave[wave_index()] = inc;
    __syncthreads();
    int before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kSampleWaves; ++w) {
        if (w < wave_index()) before += s_wave[w];
        sum += s_wave[w];
    }
    *total = sum;
    return before + inc - v;
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
    rsrc_t memory;          // the row's chunks; behind them reads give zero
    int shift;              // values before the row's first in its first chunk
    int chunk0, chunks;

    __device__ __forceinline__ Segment(const SampleArgs &a, int r, int segment, int chunks)
        : chunks(chunks) {
        const uintptr_t at = (uintptr_t)a.x + (uint64_t)r * a.stride * L::kBytes;
        shift = (int)(at & 15) / L::kBytes;
        chunk0 = segment * chunks;
        const int total = (shift + a.vocab + L::kPer - 1) / L::kPer;
        memory = __builtin_amdgcn_make_buffer_rsrc((void *)(at - shift * L::kBytes), (short)0,
                                                   16 * total, 0x00020000);
    }
    __device__ __forceinline__ u32x4 chunk(int i) const { return buf_ld16<false>(memory, 16u * (uint32_t)i); }
    // f(value, index) for every value of this lane (NaN too), as often in all lanes; what
    // is beyond the row is -inf.  U values to a round of the loop: more of them are more
    // code than is fetched while a short segment's values are on their way (two thirds of
    // the time of one row went into that), and as many registers.
    template <int U, class F>
    __device__ __forceinline__ void each(int vocab, F f) const {
        const int lane = lane_id();
        // Chunks that hold values of the row only, and all lanes have one.
        const int from = shift ? 1 : 0, to = min(chunk0 + chunks, (shift + vocab) / L::kPer);
        const int first = chunk0 + lane;
        u32x4 c0 = chunk(first), c1 = chunk(first + 64), c2 = chunk(first + 128), c3 = chunk(first + 192);
#pragma unroll 1
        for (int i0 = 0; i0 < chunks; i0 += 64) {
            u32x4 c = c0;
            c0 = c1;
            c1 = c2;
            c2 = c3;
            c3 = chunk(first + i0 + 256);
            const int at = (first + i0) * L::kPer - shift;
            if (chunk0 + i0 < from || chunk0 + i0 + 64 > to) {
#pragma unroll
                for (int e = 0; e < L::kPer; ++e)
                    if (i0 + lane >= chunks || (uint32_t)(at + e) >= (uint32_t)vocab) L::hide(c, e);
            }
            constexpr int kRound = U < L::kPer ? U : L::kPer;
#pragma unroll 1
            for (int e = 0; e < L::kPer; e += kRound) {
#pragma unroll
                for (int j = 0; j < kRound; ++j) f(L::get(c, j), at + e + j);
                if constexpr (kRound == 4 && L::kPer == 8) c = (u32x4){c[2], c[3], 0u, 0u};
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
template <int Type>
__device__ __forceinline__ SampleBorder find_border(const SampleArgs &a, const SampleRow &f, int row,
                                                    float scale, const uint64_t *own_hist,
                                                    int *s_wave_i, double *s_wave_d, double *s_far,
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
    const float place = sample_place(max, scale);
    const int bin = sample_top(place);
    const int by = its_max > -__builtin_inff() ? min(bin - (int)(uint32_t)h1, kSampleBins) : kSampleBins;
    // A wave has bins next to each other, an octave at a time.
    const int r0 = kMine * 64 * wave_index() + lane;
    if (own < 3) s_bin[own].bin = kSampleBins - 1;
    // Counts and weights of all slices fit into such integers too: a row has 2^19 values.
    uint64_t sum[kMine] = {};
    if (a.slices_n == 1) {
#pragma unroll
        for (int j = 0; j < kMine; ++j) sum[j] = own_hist[r0 + 64 * j];
    } else {
        // Several slices' loads on their way at once: each takes more than a microsecond.
        constexpr int kAtOnce = 5;
#pragma unroll 1
        for (int s0 = 0; s0 < a.slices_n; s0 += kAtOnce) {
            uint64_t v[kAtOnce][kMine];
            int off[kAtOnce];
#pragma unroll
            for (int y = 0; y < kAtOnce; ++y) {
                // (Behind the last slice the last one again, for nothing.)
                const int sl = min(s0 + y, a.slices_n - 1);
                off[y] = s0 + y < a.slices_n ? __builtin_amdgcn_readlane(by, sl) : kSampleBins;
                const uint64_t *hist = a.hist + ((int64_t)row * a.slices_n + sl) * kSampleBins;
#pragma unroll
                for (int j = 0; j < kMine; ++j)
                    v[y][j] = __hip_atomic_load(hist + max_i(r0 + 64 * j - off[y], 0),
                                                __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
#pragma unroll
            for (int y = 0; y < kAtOnce; ++y)
#pragma unroll
                for (int j = 0; j < kMine; ++j) sum[j] += r0 + 64 * j >= off[y] ? v[y][j] : 0;
        }
    }
    // Up to and with each bin; weights in units of the maximum's, up to a factor that
    // all share.
    double unit = 0x1p-24 *
                  __builtin_ldexp(exp2_64(((double)bin - (double)place - lane) * (1.0 / kSamplePerOctave)),
                                  -kMine * wave_index());
    int count[kMine], here = 0;
    double mass[kMine], here_mass = 0.0, far = 0.0;     // far: weights times bins
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
        // The last bin has what is left: its weights, below 2^-63 each, do not show, and it is
        // counted if need be.
        const bool is = r0 + 64 * j < kSampleBins - 1;
        count[j] = is ? (int)(sum[j] >> 44) : 0;
        mass[j] = is ? (double)(sum[j] & ((1ull << 44) - 1)) * unit : 0.0;
        far += mass[j] * (r0 + 64 * j);
        unit *= 0.5;
    }
    wave_scan_all<kMine>(count, mass);
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
        count[j] += here;
        mass[j] += here_mass;
        here = __builtin_amdgcn_readlane(count[j], 63);
        here_mass = lane_d(mass[j], 63);
    }
    far = wave_sum_d(far);
    __syncthreads();
    if (lane == 0) {
        s_wave_i[wave_index()] = here;
        s_wave_d[wave_index()] = here_mass;
        s_far[wave_index()] = far;
    }
    __syncthreads();
    int all_count = 0, c0 = 0;
    double all_mass = 0.0, m0 = 0.0, all_far = 0.0;
#pragma unroll
    for (int w = 0; w < kSampleWaves; ++w) {
        if (w == wave_index()) {
            c0 = all_count;
            m0 = all_mass;
        }
        all_count += s_wave_i[w];
        all_mass += s_wave_d[w];
        all_far += s_far[w];
    }
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
        count[j] += c0;
        mass[j] += m0;
    }
    // s_bin[k]: the first bin that `reached` (the last one always is): find, a barrier, tell, a
    // barrier.
    auto find = [&](int k, auto reached) {
        int r = kSampleBins - 1;
#pragma unroll
        for (int j = kMine - 1; j >= 0; --j) {
            const uint64_t are = __ballot(reached(j));
            if (are) r = kMine * 64 * wave_index() + 64 * j + __builtin_ctzll(are);
        }
        if (lane == 0) atomicMin(&s_bin[k].bin, r);
    };
    auto tell = [&](int k) {
        // Its lane tells what is there, and the one before it.
        const int r = s_bin[k].bin;
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
        }
        if (r == 0 && own == 0) {
            s_bin[k].count_before = 0;
            s_bin[k].mass_before = 0.0;
        }
    };
    int top = 0, bottom = kSampleBins - 1, above = 0, upto = 0;
    double lo = all_mass, hi = all_mass;
    if (f.top_k) {
        find(0, [&](int j) { return count[j] >= f.top_k; });
        __syncthreads();
        tell(0);
        __syncthreads();
        const SampleBin k = s_bin[0];
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
        // What a border may be off by.  A weight is off by e < 2^-20.1: the exponent, formed
        // near 24, is rounded to a multiple of 2^-19 (2^-20.5 of the weight), its power to 23
        // bits, and that cut off to 24 bits.  Where the weights before a border are p of all
        // and off by e one way, and the others the other way, they less p times the sum of
        // all are off by 2 e p (1 - p) of that sum, at most 2^-21.1 (the sum errs with
        // them); the margin is (1 + p) 2^-21.  Then for a value's place and the scale,
        // rounded to 24 bits both (ln 2 / 64 a place; more, where they are off by many).
        const double off = all_mass * (0x1p-21 + fabs((double)place) * 0x1p-24 * 0.035) +
                           all_far * 0x1p-24 * 0.035;
        const double least = f.top_p * (lo - off) - off, most = f.top_p * (hi + off) + off;
        find(1, [&](int j) { return mass[j] >= least; });
        if (!f.top_k) find(2, [&](int j) { return mass[j] >= most; });
        __syncthreads();
        tell(1);
        if (!f.top_k) tell(2);
        __syncthreads();
        const SampleBin p = s_bin[1];
        if (!f.top_k || p.bin < top) {
            top = p.bin;
            above = p.count_before;
        }
        if (!f.top_k) {
            bottom = s_bin[2].bin;
            upto = s_bin[2].count;
        }
    }
    if (bottom == kSampleBins - 1) {
        // All finite values, then.
        int n = 0;
        for (int i = wave_index(); i < a.slices_n * kSampleWaves; i += kSampleWaves)
            Segment<Type>(a, row, i, a.chunks)
                .template each<4>(a.vocab, [&](float x, int) { n += x > -__builtin_inff(); });
        n = wave_sum_i(n);
        __syncthreads();
        if (lane == 0) s_wave_i[wave_index()] = n;
        __syncthreads();
        upto = 0;
#pragma unroll
        for (int w = 0; w < kSampleWaves; ++w) upto += s_wave_i[w];
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
    __shared__ double s_wave_d[kSampleWaves], s_far[kSampleWaves];
    __shared__ int s_wave_i[kSampleWaves];
    __shared__ SampleBin s_bin[3];
    __shared__ uint32_t s_last;
    __shared__ float s_max[kSampleWaves];
    __shared__ int s_first[kSampleWaves];
    const int row = (int)blockIdx.x / a.slices_n, slice = (int)blockIdx.x % a.slices_n;
    const int lane = lane_id(), wave = wave_index();
    const SampleRow f = sample_row(a, row);
    Segment<Type> seg(a, row, slice * kSampleWaves + wave, a.chunks);
    const bool binned = !f.greedy && (f.top_k || f.by_p);
    if (binned)
        for (int i = threadIdx.x; i < kSampleBins; i += kSampleThreads) s_hist[i] = 0;
    float max = -__builtin_inff();
    seg.template each<8>(a.vocab, [&](float x, int) { max = fmaxf(max, x); });
    max = wave_max(max);
    int first = 0x7FFFFFFF;
    if (f.greedy) {
        seg.template each<8>(a.vocab, [&](float x, int i) { first = x == max ? min(first, i) : first; });
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
    if (threadIdx.x == 0)
        __hip_atomic_store(mine + 1, (uint64_t)(uint32_t)top, __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
    if (max > -__builtin_inff())
        seg.template each<8>(a.vocab, [&](float x, int) {
            const float place = sample_place(x, scale);
            const int r = top - sample_bin(place);
            // 2^24 times the weight in units of that of the bin's upper end
            const float w = exp2_(fmaf(__builtin_amdgcn_fractf(place), 1.f / kSamplePerOctave,
                                       24.f - 1.f / kSamplePerOctave));
            if (r < kSampleBins - 1)
                __hip_atomic_fetch_add(&s_hist[r], 1ull << 44 | (uint32_t)w, __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_WORKGROUP);
        });
    __syncthreads();
    if (a.slices_n > 1) {
        uint64_t *hist = a.hist + (int64_t)blockIdx.x * kSampleBins;
        for (int i = threadIdx.x; i < kSampleBins; i += kSampleThreads)
            __hip_atomic_store(hist + i, s_hist[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    wait_vm_all();
    __syncthreads();
    if (threadIdx.x == 0)
        s_last = __hip_atomic_fetch_add(a.counters + row, 1u, __ATOMIC_RELAXED,
                                        __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (s_last != (uint32_t)a.slices_n - 1) return;
    const SampleBorder b = find_border<Type>(a, f, row, scale, s_hist, s_wave_i, s_wave_d, s_far,
                                             s_bin);
    if (threadIdx.x == 0) {
        a.borders[row] = b;
        store_agent(a.counters + row, 0u);
    }
}

template <int Type>
struct SampleLds {
    uint64_t list[kSampleList];
    uint32_t count_of[kSampleKeyBins];
    unsigned long long mass_of[kSampleKeyBins];
    // Places of their own: block_scan_d reads its array behind its last barrier, so that a
    // wave may have gone on to write list_first and wave_u while another still reads wave_d.
    // (Of one array, block_scan_d's first barrier keeps its uses apart.)
    double wave_d[kSampleWaves];
    uint64_t wave_u[kSampleWaves];
    int wave_i[kSampleWaves];
    double seg[kSampleSegments + 1];
    union {
        double upto[kSampleSegments];          // of a segment's kept ones at the border
        unsigned long long quanta[kSampleSegments];
    };
    uint8_t some[kSampleSegments];             // whether the kept ones at the border have weight
    int n, place[2 * kSampleWaves];
    uint32_t last;
    int count, before, bin;
    uint64_t mass_before, border, list_first[kSampleWaves], list_end[kSampleWaves];
};
// Of k_sample_plain.
struct SamplePlainLds {
    double wave_d[kSampleWaves];
    double seg[kSampleSegments + 1];
    int place[2 * kSampleWaves];
    uint32_t last;
};

// The first thread whose place `holds`; where none does, the last that has `some`, or 0.
// One barrier after the places are known (s.place: two for each wave).
template <class Lds>
__device__ __forceinline__ int first_place(Lds &s, bool holds, bool some) {
    const uint64_t h = __ballot(holds), any = __ballot(some);
    const int base = 64 * wave_index();
    __syncthreads();
    if (lane_id() == 0) {
        s.place[wave_index()] = h ? base + (int)__builtin_ctzll(h) : 0x7FFFFFFF;
        s.place[kSampleWaves + wave_index()] = any ? base + 63 - (int)__builtin_clzll(any) : 0;
    }
    __syncthreads();
    int first = 0x7FFFFFFF, last = 0;
#pragma unroll
    for (int w = 0; w < kSampleWaves; ++w) {
        first = min(first, s.place[w]);
        last = max_i(last, s.place[kSampleWaves + w]);
    }
    return first != 0x7FFFFFFF ? first : last;
}

// The token of a row whose sums up to each segment are in s.seg: the segment, then the
// place in it.  A thread takes a few chunks next to each other.  weight_of(x) of any of the
// row's values, weight(x) as it is kept, and is_kept(x, index).  some: whether segment
// `threadIdx.x` holds any weight.  (Not what the sums up to it say: two that differ by
// nothing may be off by a rounding, and a weight may be too small to show in them.)
template <int Type, class Lds, class Weight, class Is>
__device__ __forceinline__ void draw_token(const SampleArgs &a, int row, const SampleRow &f,
                                           Lds &s, bool some, const SampleWeight &weight_of,
                                           Weight weight, Is is_kept) {
    typedef Logits<Type> L;
    const int own = threadIdx.x, segments = a.draws * kSampleWaves;
    const double total = s.seg[segments];
    // From 1 on the target is beyond every sum, so that the last weight is taken; every
    // weight is beyond a target of 0.
    const double target = f.u < 1.f ? (double)f.u * total : __builtin_inf();
    const bool holds = some && (target == 0.0 || s.seg[own + 1] > target);
    const int who = first_place(s, holds, some);
    const Segment<Type> seg(a, row, who, a.draw_chunks);
    const int per = (a.draw_chunks + kSampleThreads - 1) / kSampleThreads, first = own * per;
    auto each_kept = [&](auto take) {
#pragma unroll 1
        for (int j = 0; j < per; ++j) {
            const int in = first + j, at = (seg.chunk0 + in) * L::kPer - seg.shift;
            u32x4 c = seg.chunk(seg.chunk0 + in);
#pragma unroll 1
            for (int e = 0; e < L::kPer; e += 4) {
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float x = L::get(c, y);
                    const int i = at + e + y;
                    const bool is = in < a.draw_chunks && (uint32_t)i < (uint32_t)a.vocab &&
                                    x > -__builtin_inff() && is_kept(x, i);
                    take(i, x, is ? weight(x) : 0.0);
                }
                if constexpr (L::kPer == 8) c = (u32x4){c[2], c[3], 0u, 0u};
            }
        }
    };
    // Twice: the threads' sums, then the token by the thread that has it.
    double sum = 0.0, before = 0.0;
    int by = own;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        double at = before;
        float logit = 0.f;
        int token = 0;
        bool found = false;
        if (own == by)
            each_kept([&](int i, float x, double w) {
                at += w;
                if (!found && w > 0.0) {
                    token = i;
                    logit = x;
                    found = at > target;
                }
            });
        if (pass) {
            if (own == by) {
                a.token[row] = token;
                // (Not by its weight, which may be below the normal numbers.)
                a.logprob[row] =
                    (float)(weight_of.exponent(logit) * 0.69314718055994530942 - log_64(total));
            }
            return;
        }
        double all;
        sum = at;
        before = s.seg[who] + block_scan_d(sum, &all, s.wave_d);
        // (Where rounding leaves nobody beyond the target, the last that is kept.)
        by = first_place(s, sum > 0.0 && before + sum > target, sum > 0.0);
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

// Among values in the order of tokens, from lo to hi: the one at which a sum reaches
// `target`, by count or by weight (in units), else the last one, as s.border; what is
// before it in s.before and (if weights are summed) s.mass_before.  base: the sum before
// the first of them.  visit(f) calls f(order, weight()) for all there are.
template <class Lds, class Visit>
__device__ __forceinline__ void find_border_token(Lds &s, bool by_mass, bool summed, double base,
                                                  double unit, double target, uint64_t lo,
                                                  uint64_t hi, Visit visit) {
    const double per = 1.0 / unit;
    int before = 0;
    uint64_t mass_before = 0;
    for (;;) {
        const uint64_t range = hi - lo;
        const int shift = range < kSampleKeyBins ? 0 : 64 - 11 - __builtin_clzll(range);
        __syncthreads();
        for (int i = threadIdx.x; i < kSampleKeyBins; i += kSampleThreads) {
            s.count_of[i] = 0;
            s.mass_of[i] = 0;
        }
        __syncthreads();
        visit([&](uint64_t order, auto weight) {
            if (order < lo || order > hi) return;
            const int bin = (int)((order - lo) >> shift);
            atomicAdd(&s.count_of[bin], 1u);
            if (summed) atomicAdd(&s.mass_of[bin], (unsigned long long)__builtin_rint(weight() * per));
        });
        __syncthreads();
        // The bin at which the sum reaches the target, or the last that holds any.
        constexpr int kMine = kSampleKeyBins / kSampleThreads;
        const int r0 = kMine * (int)threadIdx.x;
        int here = 0, all_count;
        uint64_t here_mass = 0, all_mass;
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            here += (int)s.count_of[r0 + j];
            here_mass += s.mass_of[r0 + j];
        }
        const int c0 = before + block_scan_i(here, &all_count, s.wave_i);
        uint64_t m0 = 0;
        if (summed) m0 = mass_before + block_scan_d(here_mass, &all_mass, s.wave_u);
        auto reached = [&](int c, uint64_t m) {
            return by_mass ? base + (double)m * unit >= target : base + (double)c >= target;
        };
        const int who = first_place(s, here && reached(c0 + here, m0 + here_mass), here != 0);
        if ((int)threadIdx.x == who) {
            int c = c0;
            uint64_t m = m0;
#pragma unroll 1
            for (int j = 0; j < kMine; ++j) {
                const int n = (int)s.count_of[r0 + j];
                if (!n) continue;
                s.bin = r0 + j;
                s.count = n;
                s.before = c;
                s.mass_before = m;
                c += n;
                m += s.mass_of[r0 + j];
                if (reached(c, m)) break;
            }
        }
        __syncthreads();
        before = s.before;
        mass_before = s.mass_before;
        lo += (uint64_t)s.bin << shift;
        hi = min(hi, lo + ((1ull << shift) - 1));
        if (s.count == 1 || shift == 0) break;
    }
    if (threadIdx.x == 0) s.border = lo;
    __syncthreads();
    if (lo < hi)     // the only one in its bin
        visit([&](uint64_t order, auto) {
            if (order >= lo && order <= hi) s.border = order;
        });
    __syncthreads();
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
    const SampleWeight weight_of(max, f.temperature);
    const double min_p = f.min_p;
    if (!f.top_k && !f.by_p) b = {-3.402823466e38f, -3.402823466e38f, a.vocab, 0};   // all are above
    auto kept_weight = [&](float x) {
        const double w = weight_of(x);
        return w >= min_p ? w : 0.0;
    };
    auto is_listed = [&](float x) { return x >= b.bottom && !(x >= b.top); };
    const bool wide = b.listed > kSampleList;
    const bool rest = f.by_p && !f.top_k;     // the sum of all weights is needed
    uint32_t *arrived = a.counters + row;
    if (threadIdx.x == 0) s.n = 0;
    __syncthreads();
    double above = 0.0, kept = 0.0, total = 0.0;
    auto list_it = [&](float x, int i) {
        if (wide) return;
        const int at = atomicAdd(&s.n, 1);
        if (at < kSampleList) s.list[at] = sample_order<Type>(x, i);
    };
    if (rest)
        seg.template each<4>(a.vocab, [&](float x, int i) {
            const double w = weight_of(x);
            total += w;
            const double is = x >= b.top ? w : 0.0;
            above += is;
            if (min_p > 0.0) kept += is >= min_p ? is : 0.0;
            if (is_listed(x)) list_it(x, i);
        });
    else
        seg.template each<4>(a.vocab, [&](float x, int i) {
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
    if (lane == 0) {
        const int64_t at = (int64_t)blockIdx.x * kSampleWaves + wave;
        double *to = a.sums + at * kSampleSlots;
        store_agent_d(to, above);
        store_agent_d(to + 1, kept);
        store_agent_d(to + 2, total);
    }
    __syncthreads();
    int n = min(s.n, kSampleList);
    if (a.draws > 1) {
        uint64_t *list = a.list + (int64_t)blockIdx.x * kSampleList;
        for (int i = threadIdx.x; i < n; i += kSampleThreads)
            __hip_atomic_store(list + i, s.list[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (threadIdx.x == 0)
            __hip_atomic_store(a.listed + blockIdx.x, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
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

    // The border: in the order of tokens those up to this one are kept.
    uint64_t border = 0;
    const int own = (int)threadIdx.x, per_segment = a.draw_chunks * L::kPer;
    double listed_kept = 0.0;       // of the listed ones those in segment `own`
    bool listed_some = false;
    if (b.listed) {
        if (!wide && a.draws > 1) {
            // All slices' shares of the list: the n-th of all is in the share whose first is
            // the last one up to n.
            const int upto = wave_scan_i(lane < a.draws ? listed : 0);
            n = __builtin_amdgcn_readlane(upto, 63);
            for (int j0 = 64 * wave; j0 < n; j0 += kSampleThreads) {
                const int j = j0 + lane;
                int share = 0, at = 0;
                for (int i = 0; i < a.draws - 1; ++i) {
                    const int end = __builtin_amdgcn_readlane(upto, i);
                    share = j >= end ? i + 1 : share;
                    at = j >= end ? end : at;
                }
                if (j < n)
                    s.list[j] = __hip_atomic_load(
                        a.list + ((int64_t)row * a.draws + share) * kSampleList + j - at,
                        __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
        }
        if (!wide)
            for (int i = own; i < segments; i += kSampleThreads) {
                s.quanta[i] = 0;
                s.some[i] = 0;
            }
        auto visit = [&](auto f) {
            if (wide) {
                each_segment<Type>(a, row, [&](const Segment<Type> &seg, int) {
                    seg.template each<4>(a.vocab, [&](float x, int i) {
                        if (is_listed(x)) f(sample_order<Type>(x, i), [&] { return weight_of(x); });
                    });
                });
            } else {
                for (int j = own; j < n; j += kSampleThreads) {
                    const uint64_t v = s.list[j];
                    f(v, [&] { return weight_of(sample_ordered<Type>(v)); });
                }
            }
        };
        // Weights as integers, whose sums have no order: in 2^-44 of a power of two that
        // none of these reaches.
        const float largest = b.top == b.top ? b.top : max;
        const int e = max_i(__builtin_amdgcn_frexp_exp(weight_of(largest)), -900) - 44;
        const double unit = __builtin_ldexp(1.0, e);
        uint64_t lo = sample_order<Type>(largest, 0);
        border = sample_order<Type>(b.bottom, (1 << kSampleIndexBits) - 1);
        if (!wide) {
            // From the first to the last of the list: fewer passes, and fewer in one bin,
            // whose additions wait for each other.
            uint64_t first = ~0ull, last = 0;
            for (int j = own; j < n; j += kSampleThreads) {
                first = min_u64(first, s.list[j]);
                last = max_u64(last, s.list[j]);
            }
#pragma unroll 1
            for (int m = 32; m >= 1; m >>= 1) {
                first = min_u64(first, xor_u64(first, m));
                last = max_u64(last, xor_u64(last, m));
            }
            if (lane == 0) {
                s.list_first[wave] = first;
                s.list_end[wave] = last;
            }
            __syncthreads();
            lo = s.list_first[0];
            border = s.list_end[0];
#pragma unroll
            for (int w = 1; w < kSampleWaves; ++w) {
                lo = min_u64(lo, s.list_first[w]);
                border = max_u64(border, s.list_end[w]);
            }
        }
        double mass = all_weights;
        if (f.top_k || f.by_p) {
#pragma unroll 1
            for (int by_p = f.top_k ? 0 : 1; by_p <= (f.by_p ? 1 : 0); ++by_p) {
                find_border_token(s, by_p, f.by_p, by_p ? all_above : (double)b.above, unit,
                                  by_p ? (double)f.top_p * mass : (double)f.top_k, lo, border, visit);
                border = s.border;
                // (The first kept ones' weights: up to and with this one.)
                mass = all_above + (double)s.mass_before * unit +
                       weight_of(sample_ordered<Type>(border));
            }
        }
        if (wide) {
            each_segment<Type>(a, row, [&](const Segment<Type> &seg, int i) {
                double sum = 0.0;
                seg.template each<4>(a.vocab, [&](float x, int at) {
                    if (is_listed(x) && sample_order<Type>(x, at) <= border) sum += kept_weight(x);
                });
                sum = wave_sum_d(sum);
                if (lane == 0) s.upto[i] = sum;
            });
            __syncthreads();
            listed_kept = own < segments ? s.upto[own] : 0.0;
            listed_some = listed_kept > 0.0;
        } else {
            const double per = 1.0 / unit;
            for (int j = own; j < n; j += kSampleThreads) {
                const uint64_t v = s.list[j];
                const double w = v > border ? 0.0 : kept_weight(sample_ordered<Type>(v));
                if (!(w > 0.0)) continue;
                const int at = (sample_index(v) + seg.shift) / per_segment;
                s.some[at] = 1;
                atomicAdd(&s.quanta[at], (unsigned long long)__builtin_rint(w * per));
            }
            __syncthreads();
            listed_kept = own < segments ? (double)s.quanta[own] * unit : 0.0;
            listed_some = own < segments && s.some[own];
        }
    }
    double all_listed = 0.0, listed_before = 0.0;
    if (b.listed) listed_before = block_scan_d(listed_kept, &all_listed, s.wave_d);
    if (own <= segments)
        s.seg[own] = own < segments ? kept_before + listed_before : all_kept + all_listed;
    __syncthreads();
    draw_token<Type>(a, row, f, s, kept > 0.0 || listed_some, weight_of, kept_weight,
                     [&](float x, int i) {
                         return x >= b.top || sample_order<Type>(x, i) <= border;
                     });
}

// Rows without filters.
template <int Type>
__global__ __launch_bounds__(kSampleThreads, 4) void k_sample_plain(const SampleArgs a) {
    __shared__ SamplePlainLds s;
    const int row = (int)blockIdx.x / a.draws, slice = (int)blockIdx.x % a.draws;
    const int lane = lane_id(), wave = wave_index(), own = threadIdx.x;
    const SampleRow f = sample_row(a, row);
    // The segment's maximum, where it is first, and the weights in units of its own.
    {
        const Segment<Type> seg(a, row, slice * kSampleWaves + wave, a.draw_chunks);
        float max = -__builtin_inff();
        seg.template each<4>(a.vocab, [&](float x, int) { max = fmaxf(max, x); });
        max = wave_max(max);
        double sum = 0.0;
        int first = 0x7FFFFFFF;
        if (f.greedy) {
            seg.template each<4>(a.vocab, [&](float x, int i) { first = x == max ? min(first, i) : first; });
            first = wave_min_i(first);
        } else if (max > -__builtin_inff()) {
            const SampleWeight weight_of(max, f.temperature);
            seg.template each<4>(a.vocab, [&](float x, int) { sum += weight_of(x); });
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
    const SampleWeight weight_of(max, f.temperature);
    double before = 0.0;
    bool some = false;
#pragma unroll 1
    for (int j = 0; j < kEach && 64 * j < segments; ++j) {
        const int i = 64 * j + lane;
        const bool is = i < segments && its[j] > -__builtin_inff();
        const double has = is ? part[j] * weight_of(its[j]) : 0.0;
        const double inc = before + wave_scan_d(has);
        if (wave == j) some = has > 0.0;
        if (wave == 0 && i < segments) s.seg[i + 1] = inc;
        before = lane_d(inc, 63);
    }
    if (own == 0) s.seg[0] = 0.0;
    __syncthreads();
    draw_token<Type>(a, row, f, s, some, weight_of, weight_of,
                     [](float, int) { return true; });
}

}  // namespace serve
}  // namespace moe
