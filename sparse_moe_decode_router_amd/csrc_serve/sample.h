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
// Nothing is sorted as a whole.  A row is cut into slices, one workgroup each,
// which hold theirs in registers:
//   k_sample_scan   each slice's maximum and a histogram of its values over bins of
//                   1/16 in units of T ln 2: how many, and their weights to some
//                   20 bits, both in one 64-bit integer addition.
//   k_sample_draw   every slice finds from all histograms the few bins in which the
//                   filters' borders are; sums, in 64 bits, the weights above them;
//                   and lists the values in them.  The last slice of a row to
//                   finish sorts that list, finds the border, the segment (a
//                   wave's share of a slice) that holds the token, and the token.
// Bins are monotonic in the value and their counts exact, so that the list holds the
// border whatever the weights' 20 bits missed (the margin of the search covers
// that).  A row whose list would be too long (thousands of equal logits at the
// border) is finished by its last workgroup with a radix search over the values'
// bits, from memory, 8 bits a pass: slower, and right for everything.
#pragma once

#include "serve_common.h"

namespace moe {
namespace serve {

constexpr int kSampleThreads = 512;
constexpr int kSampleWaves = kSampleThreads / 64;
constexpr int kSampleChunks = 16;       // 16-byte chunks of a thread, in registers
constexpr int kSampleMaxSlices = 16;
constexpr int kSampleBins = 1024;       // the last one takes all that is below
constexpr float kSamplePerOctave = 16.f;
constexpr int kSampleList = 4096;       // values at the border of a row
constexpr int kSampleSlots = 3;         // sums of a segment: above, above and kept, the rest

struct SampleSlice {
    float max;         // -inf: nothing to draw
    int32_t first;     // index of the first value that is the maximum
    int32_t bin;       // of the maximum
    int32_t count;     // values above -inf
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
    double *sums;             // [rows][slices][waves][kSampleSlots]
    uint64_t *list;           // [rows][kSampleList]
    uint32_t *counters;       // [rows][2]: arrivals, values in the list
    int64_t stride;           // of rows, in elements
    int32_t rows, vocab, slices_n;
    int32_t chunks;           // of a wave's segment
};

enum { kSampleF32 = 3 };   // beside MOE_BF16 and MOE_FP16

__device__ __forceinline__ int max_i(int a, int b) { return a > b ? a : b; }

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
    static __device__ __forceinline__ float load(const char *row, int i) {
        if constexpr (Type == kSampleF32) return *((const float *)row + i);
        const uint32_t h = *((const uint16_t *)row + i);
        if constexpr (Type == 0) return Bf16::lo(h);
        return Fp16::lo(h);
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

// A value's bin, monotonic in it: the place in units of T ln 2 / 16, rounded down.
__device__ __forceinline__ float sample_scale(float temperature) {
    return fminf(kSamplePerOctave * kLog2e / temperature, 0x1p90f);
}
__device__ __forceinline__ float sample_place(float x, float scale) {
    return fminf(fmaxf(x * scale, -0x1p29f), 0x1p29f);
}
__device__ __forceinline__ int sample_bin(float place) { return (int)__builtin_floorf(place); }

// 2^y for y <= 0, to some 2^-44: the power series of 2^r, |r| <= 1/2, up to the eleventh power.
__device__ __forceinline__ double exp2_64(double y) {
    y = fmax(y, -1100.0);
    const double n = __builtin_rint(y), r = (y - n) * 0.69314718055994530942;
    double p = 1.0 / 39916800;
    p = fma(p, r, 1.0 / 3628800);
    p = fma(p, r, 1.0 / 362880);
    p = fma(p, r, 1.0 / 40320);
    p = fma(p, r, 1.0 / 5040);
    p = fma(p, r, 1.0 / 720);
    p = fma(p, r, 1.0 / 120);
    p = fma(p, r, 1.0 / 24);
    p = fma(p, r, 1.0 / 6);
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    return __builtin_ldexp(p, (int)n);
}
// c: log2(e) / T.  The maximum has weight 1, also where it is infinite.
__device__ __forceinline__ double sample_weight(float x, float max, double c) {
    if (x == max) return 1.0;
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

__device__ __forceinline__ double shfl_up_d(double v, int d) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __shfl_up((uint32_t)b, d), hi = __shfl_up((uint32_t)(b >> 32), d);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum_d(double v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = __shfl_xor((uint32_t)b, m), hi = __shfl_xor((uint32_t)(b >> 32), m);
        v += __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
    }
    return v;
}
// Sum of the threads' values before this one, and of all.
__device__ __forceinline__ double block_scan_d(double v, double *total, double *s_wave) {
    double inc = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double o = shfl_up_d(inc, d);
        if (lane_id() >= d) inc += o;
    }
    __syncthreads();
    if (lane_id() == 63) s_wave[wave_index()] = inc;
    __syncthreads();
    double before = 0.0, all = 0.0;
#pragma unroll
    for (int w = 0; w < kSampleWaves; ++w) {
        if (w < wave_index()) before += s_wave[w];
        all += s_wave[w];
    }
    *total = all;
    // (Not inc - v: the sum of what is before has its own rounding.)
    const double prev = shfl_up_d(inc, 1);
    return before + (lane_id() ? prev : 0.0);
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
    u32x4 c[kSampleChunks];

    __device__ __forceinline__ Segment(const SampleArgs &a, int r, int segment) {
        const uintptr_t at = (uintptr_t)a.x + (uint64_t)r * a.stride * L::kBytes;
        row = (const char *)at;
        shift = (int)(at & 15) / L::kBytes;
        chunks = a.chunks;
        chunk0 = segment * chunks;
        total = (shift + a.vocab + L::kPer - 1) / L::kPer;
    }
    __device__ __forceinline__ void load() {
        const char *base = row - shift * L::kBytes;
#pragma unroll
        for (int i = 0; i < kSampleChunks; ++i)
            if (64 * i < chunks)
                c[i] = ld16(base + 16 * (int64_t)min(chunk0 + min(64 * i + lane_id(), chunks - 1),
                                                     total - 1));
    }
    // f(value, index) for every value of this lane; those that are none are -inf.
    template <class F>
    __device__ __forceinline__ void each(int vocab, F f) const {
#pragma unroll
        for (int i = 0; i < kSampleChunks; ++i) {
            if (64 * i < chunks) {
                const int in = 64 * i + lane_id(), i0 = (chunk0 + in) * L::kPer - shift;
#pragma unroll
                for (int e = 0; e < L::kPer; ++e) {
                    const float x = L::get(c[i], e);
                    const bool real = in < chunks && (uint32_t)(i0 + e) < (uint32_t)vocab && x == x;
                    f(real ? x : -__builtin_inff(), i0 + e);
                }
            }
        }
    }
};

template <int Type>
__global__ __launch_bounds__(kSampleThreads) void k_sample_scan(const SampleArgs a) {
    __shared__ uint64_t s_hist[kSampleBins];
    __shared__ float s_max[kSampleWaves];
    __shared__ int s_first[kSampleWaves], s_count[kSampleWaves];
    const int row = (int)blockIdx.x / a.slices_n, slice = (int)blockIdx.x % a.slices_n;
    const int lane = lane_id(), wave = wave_index();
    const SampleRow f = sample_row(a, row);
    Segment<Type> seg(a, row, slice * kSampleWaves + wave);
    seg.load();
    const bool binned = !f.greedy && (f.top_k || f.by_p);
    if (binned)
        for (int i = threadIdx.x; i < kSampleBins; i += kSampleThreads) s_hist[i] = 0;
    float max = -__builtin_inff();
    int count = 0;
    seg.each(a.vocab, [&](float x, int) {
        max = fmaxf(max, x);
        count += x > -__builtin_inff();
    });
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) max = fmaxf(max, __shfl_xor(max, m));
    count = wave_sum_i(count);
    int first = 0x7FFFFFFF;
    if (f.greedy) {
        seg.each(a.vocab, [&](float x, int i) { first = x == max ? min(first, i) : first; });
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1) first = min(first, __shfl_xor(first, m));
    }
    if (lane == 0) {
        s_max[wave] = max;
        s_first[wave] = first;
        s_count[wave] = count;
    }
    __syncthreads();
    max = s_max[0];
#pragma unroll
    for (int w = 1; w < kSampleWaves; ++w) max = fmaxf(max, s_max[w]);
    first = 0x7FFFFFFF;
    count = 0;
#pragma unroll
    for (int w = 0; w < kSampleWaves; ++w) {
        first = s_max[w] == max ? min(first, s_first[w]) : first;
        count += s_count[w];
    }
    const float scale = sample_scale(f.temperature);
    const int top = sample_bin(sample_place(max, scale));
    if (threadIdx.x == 0) {
        const SampleSlice out = {max, first, top, count};
        a.slices[blockIdx.x] = out;
    }
    if (!binned || max == -__builtin_inff()) return;
    seg.each(a.vocab, [&](float x, int) {
        if (x == -__builtin_inff()) return;
        const float place = sample_place(x, scale);
        const int bin = sample_bin(place);
        // 2^24 times the weight in units of that of the bin's upper end
        const float w = exp2_((place - (float)bin - 1.f) * (1.f / kSamplePerOctave)) * 0x1p24f;
        const uint64_t add = 1ull << 44 | (uint64_t)(uint32_t)w;
        __hip_atomic_fetch_add(&s_hist[min(top - bin, kSampleBins - 1)], add, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_WORKGROUP);
    });
    __syncthreads();
    uint64_t *hist = a.hist + (int64_t)blockIdx.x * kSampleBins;
    for (int i = threadIdx.x; i < kSampleBins; i += kSampleThreads) hist[i] = s_hist[i];
}

// What the slices of a row agree on: bins above `top` are kept by the filters, those
// below `bottom` are not, and the border is among the values between.
struct SampleBorder {
    int top, bottom;
    int above, listed;    // values above, and from top to bottom
};

// Merged histograms in LDS: counts and weights up to and with each bin.
struct SampleMerged {
    int count[kSampleBins];
    float mass[kSampleBins];
};

__device__ __forceinline__ SampleBorder find_border(const SampleArgs &a, const SampleRow &f, int row,
                                                    float max, float scale, SampleMerged &s,
                                                    int *s_wave_i, double *s_wave_d) {
    // Two bins of each thread, next to each other.
    const float place = sample_place(max, scale);
    const int bin = sample_bin(place), r0 = 2 * (int)threadIdx.x;
    int count[2] = {0, 0}, values = 0;
    uint64_t mass[2] = {0, 0};
    for (int sl = 0; sl < a.slices_n; ++sl) {
        const SampleSlice &from = a.slices[row * a.slices_n + sl];
        if (from.max == -__builtin_inff()) continue;
        values += from.count;
        const uint64_t *hist = a.hist + (int64_t)(row * a.slices_n + sl) * kSampleBins;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int at = r0 + j - (bin - from.bin);
            if (at < 0 || r0 + j == kSampleBins - 1) continue;
            count[j] += (int)(hist[at] >> 44);
            mass[j] += hist[at] & ((1ull << 44) - 1);
        }
    }
    double m[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
        m[j] = (double)mass[j] * 0x1p-24 *
               (double)exp2_(((float)(bin + 1) - place - (float)(r0 + j)) * (1.f / kSamplePerOctave));
    int all_count;
    double all_mass;
    const int c0 = block_scan_i(count[0] + count[1], &all_count, s_wave_i);
    const double m0 = block_scan_d(m[0] + m[1], &all_mass, s_wave_d);
    // The last bin has what is left; its weights, 2^-63 each, do not show.
    s.count[r0] = c0 + count[0];
    s.count[r0 + 1] = r0 + 1 == kSampleBins - 1 ? values : c0 + count[0] + count[1];
    s.mass[r0] = (float)(m0 + m[0]);
    s.mass[r0 + 1] = (float)(m0 + m[0] + m[1]);
    __syncthreads();
    // The first bin up to which `least` holds.
    auto first_bin = [&](auto least) {
        int lo = -1, hi = kSampleBins - 1;    // (the last one always is one)
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (least(mid)) hi = mid;
            else lo = mid;
        }
        return hi;
    };
    SampleBorder b;
    b.top = 0;
    b.bottom = kSampleBins - 1;
    float lo = (float)all_mass, hi = lo;
    if (f.top_k) {
        b.bottom = first_bin([&](int r) { return s.count[r] >= f.top_k; });
        b.top = b.bottom;
        lo = b.bottom ? s.mass[b.bottom - 1] : 0.f;
        hi = s.mass[b.bottom];
    }
    if (f.by_p) {
        // What the weights may be off by: their place is rounded in 32 bits, then their
        // power and their 24 bits, and the sums.
        const float off = 0x1p-16f + (fabsf(place) + (float)kSampleBins) * 0x1p-24f;
        const float least = f.top_p * lo * (1.f - off), most = f.top_p * hi * (1.f + off);
        const int p_top = first_bin([&](int r) { return s.mass[r] * (1.f + off) >= least; });
        const int p_bottom = first_bin([&](int r) { return s.mass[r] * (1.f - off) >= most; });
        b.top = f.top_k ? min(b.top, p_top) : p_top;
        b.bottom = f.top_k ? b.bottom : p_bottom;
    }
    b.above = b.top ? s.count[b.top - 1] : 0;
    b.listed = s.count[b.bottom] - b.above;
    return b;
}

// Sorts n (a power of two) 64-bit keys in LDS.
__device__ __forceinline__ void sort_keys(uint64_t *s, int n) {
    for (int size = 2; size <= n; size <<= 1)
        for (int by = size >> 1; by > 0; by >>= 1) {
            __syncthreads();
            for (int t = threadIdx.x; t < n >> 1; t += kSampleThreads) {
                const int i = 2 * t - (t & (by - 1)), j = i + by;
                const uint64_t x = s[i], y = s[j];
                const bool up = (i & size) == 0;
                if ((x > y) == up) {
                    s[i] = y;
                    s[j] = x;
                }
            }
        }
    __syncthreads();
}

template <int Type>
struct SampleLds {
    union {
        SampleMerged merged;
        uint64_t list[kSampleList];
        struct {
            uint32_t count[256];
            unsigned long long mass[256];
        } radix;
    };
    double wave_d[kSampleWaves];
    int wave_i[kSampleWaves];
    double seg[kSampleMaxSlices * kSampleWaves + 1];
    double upto[kSampleList];    // weights of what is kept of the list, up to and with each
    int n, found;
    uint32_t last;
    int token;
    double weight, mass;
};

// The row's token among the thread's n values from i0 on: `kept(x, i)` gives a value's
// weight, or zero.  base: the sum before the first thread's; all of the workgroup.
template <int Type, class Kept>
__device__ __forceinline__ void draw_in_order(const SampleArgs &a, const char *row, int i0, int n,
                                              double base, double target, SampleLds<Type> &s,
                                              Kept kept) {
    typedef Logits<Type> L;
    double sum = 0.0;
    int last = -1;
    double last_w = 0.0;
    for (int i = i0; i < i0 + n; ++i) {
        const double w = kept(L::load(row, i), i);
        sum += w;
        if (w > 0.0) {
            last = i;
            last_w = w;
        }
    }
    double all;
    const double before = base + block_scan_d(sum, &all, s.wave_d);
    // The first thread whose sum goes beyond the target; where rounding leaves none,
    // the last value that is kept.
    if (threadIdx.x == 0) s.found = 0x7FFFFFFF;
    __syncthreads();
    if (last >= 0 && before + sum > target) atomicMin(&s.found, (int)threadIdx.x);
    __syncthreads();
    int who = s.found;
    __syncthreads();
    if (who == 0x7FFFFFFF) {
        if (threadIdx.x == 0) s.found = -1;
        __syncthreads();
        if (last >= 0) atomicMax(&s.found, (int)threadIdx.x);
        __syncthreads();
        who = s.found;
    }
    if ((int)threadIdx.x == who) {
        double at = before;
        int token = last;
        double weight = last_w;
        for (int i = i0; i < i0 + n; ++i) {
            const double w = kept(L::load(row, i), i);
            at += w;
            if (w > 0.0 && at > target) {
                token = i;
                weight = w;
                break;
            }
        }
        s.token = token;
        s.weight = weight;
    }
    __syncthreads();
}

// A row by radix search over its values' keys, from memory: any row, with one
// workgroup.  Weights are summed as integers of 44 bits here.
template <int Type>
__device__ __forceinline__ void draw_by_radix(const SampleArgs &a, const SampleRow &f, int row, float max, double c,
                              SampleLds<Type> &s) {
    typedef Logits<Type> L;
    const char *x = (const char *)a.x + (uint64_t)row * a.stride * L::kBytes;
    const int per = (a.vocab + kSampleThreads - 1) / kSampleThreads;
    const int i0 = min((int)threadIdx.x * per, a.vocab), n = min(per, a.vocab - i0);
    const uint32_t none = sample_key(-__builtin_inff());
    auto key_of = [&](float v) { return v == v ? sample_key(v) : none; };
    auto weight_of = [&](uint32_t key) {
        return key == none ? 0.0 : sample_weight(sample_value(key), max, c);
    };
    // Among keys up to `limit`: the key at which the count, or the weights, reach the
    // target, and what is before it.
    struct Border {
        uint32_t key;
        int before, count;           // values before it, and equal to it
        uint64_t mass;               // weights before it
    };
    auto search = [&](bool by_mass, double target, uint32_t limit) {
        Border b = {0, 0, 0, 0};
#pragma unroll 1
        for (int shift = 24; shift >= 0; shift -= 8) {
            __syncthreads();
            for (int i = threadIdx.x; i < 256; i += kSampleThreads) {
                s.radix.count[i] = 0;
                s.radix.mass[i] = 0;
            }
            __syncthreads();
            for (int i = threadIdx.x; i < a.vocab; i += kSampleThreads) {
                const uint32_t key = key_of(L::load(x, i));
                if (key > limit || key == none || ((uint64_t)(key ^ b.key) >> (shift + 8)) != 0) continue;
                atomicAdd(&s.radix.count[key >> shift & 255], 1u);
                atomicAdd(&s.radix.mass[key >> shift & 255],
                          (unsigned long long)(weight_of(key) * 0x1p44));
            }
            __syncthreads();
            // (Every thread walks the 256 sums: it is the same walk for all.)
            int d = 0, last = -1;
            int before = b.before;
            uint64_t mass = b.mass;
            Border at = b;
            for (d = 0; d < 256; ++d) {
                const int count = (int)s.radix.count[d];
                if (!count) continue;
                const uint64_t m = s.radix.mass[d];
                last = d;
                at.before = before;
                at.count = count;
                at.mass = mass;
                if (by_mass ? (double)(mass + m) >= target : (double)(before + count) >= target)
                    break;
                before += count;
                mass += m;
            }
            at.key = b.key | (uint32_t)max_i(last, 0) << shift;
            b = at;
        }
        return b;
    };
    uint32_t key = none - 1;          // kept: smaller keys, and `equal` of this one
    int equal = 0x7FFFFFFF;
    uint64_t mass = 0;
    if (f.top_k) {
        const Border b = search(false, (double)f.top_k, none - 1);
        key = b.key;
        equal = min(b.count, f.top_k - b.before);
        mass = b.mass + (uint64_t)equal * (uint64_t)(weight_of(key) * 0x1p44);
    } else if (f.by_p) {
        // All weights: a search that nothing stops ends with them.
        const Border b = search(true, 0x1p70, none - 1);
        mass = b.mass + (uint64_t)b.count * (uint64_t)(weight_of(b.key) * 0x1p44);
    }
    if (f.by_p) {
        const double target = (double)f.top_p * (double)mass;
        const Border b = search(true, target, key);
        const double w = (double)(uint64_t)(weight_of(b.key) * 0x1p44);
        const double more = w > 0.0 ? __builtin_ceil((target - (double)b.mass) / w) : 0x1p31;
        const int n_eq = (int)fmin(fmax(more, 1.0), (double)b.count);
        equal = b.key == key ? min(equal, n_eq) : n_eq;
        key = b.key;
    }
    // Equal ones are kept by index.
    int mine = 0, all;
    for (int i = i0; i < i0 + n; ++i) mine += key_of(L::load(x, i)) == key;
    int rank = block_scan_i(mine, &all, s.wave_i);
    const int rank0 = rank;
    double sum = 0.0;
    auto kept = [&](float v, int i) {
        if (i == i0) rank = rank0;
        const uint32_t k = key_of(v);
        if (k > key || (k == key && rank++ >= equal)) return 0.0;
        const double w = weight_of(k);
        return w >= (double)f.min_p ? w : 0.0;
    };
    for (int i = i0; i < i0 + n; ++i) sum += kept(L::load(x, i), i);
    double total;
    block_scan_d(sum, &total, s.wave_d);
    draw_in_order<Type>(a, x, i0, n, 0.0, (double)f.u * total, s, kept);
    if (threadIdx.x == 0) s.mass = total;
    __syncthreads();
}

template <int Type>
__global__ __launch_bounds__(kSampleThreads) void k_sample_draw(const SampleArgs a) {
    typedef Logits<Type> L;
    __shared__ SampleLds<Type> s;
    const int row = (int)blockIdx.x / a.slices_n, slice = (int)blockIdx.x % a.slices_n;
    const int lane = lane_id(), wave = wave_index();
    const SampleRow f = sample_row(a, row);
    float max = -__builtin_inff();
    for (int i = 0; i < a.slices_n; ++i) max = fmaxf(max, a.slices[row * a.slices_n + i].max);
    if (max == -__builtin_inff() || f.greedy) {
        if (slice == 0 && threadIdx.x == 0) {
            int token = max == -__builtin_inff() ? -1 : 0x7FFFFFFF;
            for (int i = 0; i < a.slices_n; ++i) {
                const SampleSlice &from = a.slices[row * a.slices_n + i];
                if (token >= 0 && from.max == max) token = min(token, from.first);
            }
            a.token[row] = token;
            a.logprob[row] = token < 0 ? -__builtin_inff() : 0.f;
        }
        return;
    }
    Segment<Type> seg(a, row, slice * kSampleWaves + wave);
    seg.load();
    const float scale = sample_scale(f.temperature);
    const double c = 1.44269504088896340736 / (double)f.temperature;
    const int bin0 = sample_bin(sample_place(max, scale));
    auto bin_of = [&](float x) {
        return min(bin0 - sample_bin(sample_place(x, scale)), kSampleBins - 1);
    };
    SampleBorder b = {kSampleBins, -1, a.vocab, 0};   // no border: all are above it
    if (f.top_k || f.by_p) b = find_border(a, f, row, max, scale, s.merged, s.wave_i, s.wave_d);
    const bool radix = b.listed > kSampleList;
    const bool rest = f.by_p && !f.top_k;     // the sum of all weights is needed
    uint32_t *arrived = a.counters + 2 * row, *listed = arrived + 1;
    uint64_t *list = a.list + (int64_t)row * kSampleList;
    if (!radix) {
        __syncthreads();      // the merged histogram makes room for the list
        if (threadIdx.x == 0) s.n = 0;
        __syncthreads();
        double above = 0.0, kept = 0.0, below = 0.0;
        seg.each(a.vocab, [&](float x, int i) {
            if (x == -__builtin_inff()) return;
            const int r = bin_of(x);
            if (r < b.top || rest) {
                const double w = sample_weight(x, max, c);
                const bool is = r < b.top;
                above += is ? w : 0.0;
                kept += is && w >= (double)f.min_p ? w : 0.0;
                below += is ? 0.0 : w;
            }
            if (r >= b.top && r <= b.bottom) {
                const int at = atomicAdd(&s.n, 1);
                if (at < kSampleList) s.list[at] = (uint64_t)sample_key(x) << 32 | (uint32_t)i;
            }
        });
        above = wave_sum_d(above);
        kept = wave_sum_d(kept);
        below = wave_sum_d(below);
        if (lane == 0) {
            double *to = a.sums + ((int64_t)blockIdx.x * kSampleWaves + wave) * kSampleSlots;
            store_agent_d(to, above);
            store_agent_d(to + 1, kept);
            store_agent_d(to + 2, below);
        }
        __syncthreads();
        const int mine = min(s.n, kSampleList);
        if (mine) {
            if (threadIdx.x == 0)
                s.found = (int)__hip_atomic_fetch_add(listed, (uint32_t)mine, __ATOMIC_RELAXED,
                                                      __HIP_MEMORY_SCOPE_AGENT);
            __syncthreads();
            const int at = s.found;
            for (int i = threadIdx.x; i < mine; i += kSampleThreads)
                if (at + i < kSampleList)
                    __hip_atomic_store(list + at + i, s.list[i], __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    wait_vm_all();
    __syncthreads();
    if (threadIdx.x == 0)
        s.last = __hip_atomic_fetch_add(arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (s.last != (uint32_t)a.slices_n - 1) return;
    if (threadIdx.x == 0) store_agent(arrived, 0u);

    // The last workgroup of the row.
    auto write = [&]() {
        if (threadIdx.x == 0) {
            a.token[row] = s.token;
            a.logprob[row] = (float)log(s.weight / s.mass);
        }
    };
    if (radix) {
        draw_by_radix<Type>(a, f, row, max, c, s);
        write();
        return;
    }
    const int segments = a.slices_n * kSampleWaves;
    const double *sums = a.sums + (int64_t)row * segments * kSampleSlots;
    double above = 0.0, kept = 0.0, below = 0.0;
    if ((int)threadIdx.x < segments) {
        above = load_agent_d(sums + threadIdx.x * kSampleSlots);
        kept = load_agent_d(sums + threadIdx.x * kSampleSlots + 1);
        below = load_agent_d(sums + threadIdx.x * kSampleSlots + 2);
    }
    double all_above, all_below, all_kept;
    block_scan_d(above, &all_above, s.wave_d);
    block_scan_d(below, &all_below, s.wave_d);
    const double kept_before = block_scan_d(kept, &all_kept, s.wave_d);
    // The list, sorted; and how much of it is kept.
    int n = 0, n2 = 2;
    uint64_t border = 0;                 // values up to this one are kept
    if (b.listed) {
        n = b.listed;
        while (n2 < n) n2 <<= 1;
        for (int i = threadIdx.x; i < n2; i += kSampleThreads)
            s.list[i] = i < n ? __hip_atomic_load(list + i, __ATOMIC_RELAXED,
                                                  __HIP_MEMORY_SCOPE_AGENT)
                              : ~0ull;
        if (threadIdx.x == 0) store_agent(listed, 0u);
        sort_keys(s.list, n2);
    }
    const int per = n2 / kSampleThreads > 0 ? n2 / kSampleThreads : 1, j0 = (int)threadIdx.x * per;
    auto weight_at = [&](int j) {
        return j < n ? sample_weight(sample_value((uint32_t)(s.list[j] >> 32)), max, c) : 0.0;
    };
    int take = n;
    if (f.top_k) take = min(n, f.top_k - b.above);
    if (f.by_p) {
        double sum = 0.0, all;
        for (int j = j0; j < min(j0 + per, take); ++j) sum += weight_at(j);
        double before = all_above + block_scan_d(sum, &all, s.wave_d);
        const double target = (double)f.top_p * (rest ? all_above + all_below : all_above + all);
        int count = 0, some;
        for (int j = j0; j < min(j0 + per, take); ++j) {
            count += before < target;
            before += weight_at(j);
        }
        block_scan_i(count, &some, s.wave_i);
        take = max_i(some, b.above ? 0 : 1);
    }
    if (take) border = s.list[take - 1];
    __syncthreads();
    // What is kept of it, by index.
    n = take;
    n2 = 2;
    while (n2 < n) n2 <<= 1;
    for (int i = threadIdx.x; i < n2; i += kSampleThreads)
        s.list[i] = i < n ? s.list[i] << 32 | s.list[i] >> 32 : ~0ull;
    sort_keys(s.list, n2);
    auto weight_by_index = [&](int j) {
        if (j >= n) return 0.0;
        const double w = sample_weight(sample_value((uint32_t)s.list[j]), max, c);
        return w >= (double)f.min_p ? w : 0.0;
    };
    const int each = n2 / kSampleThreads > 0 ? n2 / kSampleThreads : 1, k0 = (int)threadIdx.x * each;
    double sum = 0.0, all_listed;
    for (int j = k0; j < min(k0 + each, n); ++j) sum += weight_by_index(j);
    double before = block_scan_d(sum, &all_listed, s.wave_d);
    for (int j = k0; j < min(k0 + each, n); ++j) {
        before += weight_by_index(j);
        s.upto[j] = before;
    }
    const double total = all_kept + all_listed;
    const double target = (double)f.u * total;
    if (threadIdx.x == 0) {
        s.found = 0x7FFFFFFF;
        s.mass = total;
    }
    __syncthreads();
    // The first of n places that `holds`; where none does, the last that `some`.
    auto first_of = [&](int n, auto holds, auto some) {
        for (int j = threadIdx.x; j < n; j += kSampleThreads)
            if (holds(j)) {
                atomicMin(&s.found, j);
                break;
            }
        __syncthreads();
        int who = s.found;
        __syncthreads();
        if (who == 0x7FFFFFFF) {
            if (threadIdx.x == 0) s.found = 0;
            __syncthreads();
            for (int j = threadIdx.x; j < n; j += kSampleThreads)
                if (some(j)) atomicMax(&s.found, j);
            __syncthreads();
            who = s.found;
        }
        return who;
    };
    if (!b.above) {
        // Nothing but the list.
        const int who =
            first_of(n, [&](int j) { return s.upto[j] > target && weight_by_index(j) > 0.0; },
                     [&](int j) { return weight_by_index(j) > 0.0; });
        if (threadIdx.x == 0) {
            s.token = (int)(s.list[who] >> 32);
            s.weight = weight_by_index(who);
        }
        write();
        return;
    }
    // The segment: what is above the border before it, and the listed ones with lower
    // indexes than its first.
    const int per_segment = a.chunks * L::kPer;
    if ((int)threadIdx.x <= segments) {
        const int index = (int)threadIdx.x < segments ? (int)threadIdx.x * per_segment - seg.shift
                                                      : 0x7FFFFFFF;
        int lo = -1, hi = n;       // the first listed one from `index` on
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if ((int)(s.list[mid] >> 32) >= index) hi = mid;
            else lo = mid;
        }
        s.seg[threadIdx.x] = ((int)threadIdx.x < segments ? kept_before : all_kept) +
                             (hi ? s.upto[hi - 1] : 0.0);
    }
    __syncthreads();
    const int who = first_of(
        segments, [&](int j) { return s.seg[j + 1] > target && s.seg[j + 1] > s.seg[j]; },
        [&](int j) { return s.seg[j + 1] > s.seg[j]; });
    const int from = max_i(who * per_segment - seg.shift, 0);
    const int to = min((who + 1) * per_segment - seg.shift, a.vocab);
    const int share = (to - from + kSampleThreads - 1) / kSampleThreads;
    const int i0 = min(from + (int)threadIdx.x * share, to), count = min(share, to - i0);
    draw_in_order<Type>(a, seg.row, i0, count, s.seg[who], target, s, [&](float x, int i) {
        if (!(x > -__builtin_inff())) return 0.0;
        const int r = bin_of(x);
        if (r > b.bottom && r >= b.top) return 0.0;
        if (r >= b.top && !(take && ((uint64_t)sample_key(x) << 32 | (uint32_t)i) <= border))
            return 0.0;
        const double w = sample_weight(x, max, c);
        return w >= (double)f.min_p ? w : 0.0;
    });
    write();
}

}  // namespace serve
}  // namespace moe
