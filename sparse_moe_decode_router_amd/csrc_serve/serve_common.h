// serve_common.h - device helpers shared by the serving kernels: the two
// 16-bit compute types, e4m3 conversion, the view of the paged cache, and the
// visible blocks of a sequence.
#pragma once

#include "device_common.h"

namespace moe {
namespace serve {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A running maximum before any score was seen: the lowest finite value, so that
// differences from it are never NaN and every score is above it.  Scores are in
// units of log 2.
constexpr float kNoMax = -0x1.fffffep+127f;

// Compute types.  kOff: weights are held as 2^(s - max + kOff), kSlack: how far
// a score may exceed the running maximum before the accumulators are rescaled
// (both in units of log 2; the factor cancels in the end).  fp16 holds weights
// down to 2^-24 only, so they are lifted by 2^10: what is lost is below 2^-34
// of the largest weight, and 2^(10 + 4) is still in range.
struct Bf16 {
    typedef bf16x8 v8;
    static constexpr float kOff = 0.f, kSlack = 8.f;
    static __device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a),
                                                       __builtin_bit_cast(v8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8, a),
                                                       __builtin_bit_cast(v8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) { return bf16x2_rne(a, b); }
    static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
    static __device__ __forceinline__ float hi(uint32_t w) {
        return __uint_as_float(w & 0xFFFF0000u);
    }
    // Codes 2h, 2h + 1 of a dword of four e4m3 codes; exact.
    template <bool H>
    static __device__ __forceinline__ uint32_t from_e4m3(uint32_t w) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, H));
    }
    // True for the infinities and NaN (either half).
    static __device__ __forceinline__ bool odd(uint32_t h) { return (h & 0x7F80u) == 0x7F80u; }
    static __device__ __forceinline__ bool nan(uint32_t h) { return (h & 0x7FFFu) > 0x7F80u; }
    static constexpr uint32_t kOne = 0x3F80u;
};

struct Fp16 {
    typedef f16x8 v8;
    static constexpr float kOff = 10.f, kSlack = 4.f;
    static __device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a),
                                                      __builtin_bit_cast(v8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8, a),
                                                      __builtin_bit_cast(v8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, f16x2));
    }
    static __device__ __forceinline__ float lo(uint32_t w) {
        return (float)__builtin_bit_cast(f16x2, w)[0];
    }
    static __device__ __forceinline__ float hi(uint32_t w) {
        return (float)__builtin_bit_cast(f16x2, w)[1];
    }
    template <bool H>
    static __device__ __forceinline__ uint32_t from_e4m3(uint32_t w) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, H));
    }
    static __device__ __forceinline__ bool odd(uint32_t h) { return (h & 0x7C00u) == 0x7C00u; }
    static __device__ __forceinline__ bool nan(uint32_t h) { return (h & 0x7FFFu) > 0x7C00u; }
    static constexpr uint32_t kOne = 0x3C00u;
};

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_(float x) { return __builtin_amdgcn_logf(x); }

// The arguments of both attention kernels.
struct AttnArgs {
    const void *k, *v;         // the layer's [pages][kv_heads][page][head_dim]
    const int32_t *tables, *lengths;
    const float *k_scale, *v_scale;
    const void *q;
    const int32_t *cu;         // prompt only
    void *out;
    float *lse;
    float *part;               // partial results of split rows
    uint32_t *counters;
    int64_t q_token, q_head;   // strides of q in elements
    float scale;               // of the scores, times log2(e)
    int32_t batch, tokens, pages, cols, page_log2, kv_heads, group, head_groups;
    int32_t window, sinks;
    int32_t split;             // decode: units aimed at per kv head; prompt: most splits
    int32_t units;             // prompt: equal shares per kv head (0: row tiles)
    int32_t row_tiles;         // prompt: most of them that there are counters for
};

// Blocks of 2^L keys that a row at the last position of n sees: the first
// `sb` blocks of the sequence hold its sinks, the others run from block `wb`
// to the end.  The two never overlap.
struct Visible {
    int sb, wb, total;
};
template <int L>
__device__ __forceinline__ Visible visible(int n, int first, int sinks) {
    // first: the first position of the window (0: no window)
    const int end = (n + (1 << L) - 1) >> L;
    Visible v;
    v.sb = first > 0 ? min(((min(sinks, first) + (1 << L) - 1) >> L), end) : 0;
    v.wb = max(first >> L, v.sb);
    v.total = v.sb + max(0, end - v.wb);
    return v;
}
__device__ __forceinline__ int visible_block(const Visible &v, int i) {
    return i < v.sb ? i : i - v.sb + v.wb;
}

__device__ __forceinline__ int wave_sum_i(int v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
    return v;
}

// Dwords of 4-byte alignment, read as one wide load.
template <int N>
struct Words {
    typedef uint32_t type __attribute__((ext_vector_type(N), aligned(4)));
};
template <int N>
__device__ __forceinline__ void load_words(uint32_t *r, const void *p) {
    if constexpr (N > 4) {
        load_words<4>(r, p);
        load_words<N - 4>(r + 4, (const uint32_t *)p + 4);
    } else if constexpr (N == 1) {
        r[0] = *(const uint32_t *)p;
    } else {
        const typename Words<N>::type w = *(const typename Words<N>::type *)p;
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = w[i];
    }
}

// The factor of a part whose maximum is `by` above the joined one (at most 0).
// Never zero: an infinity stays one, since a weight is positive, however small.
__device__ __forceinline__ float part_factor(float by) { return fmaxf(exp2_(by), 0x1p-149f); }

// Which of two values are +inf (sign 0) or -inf (sign 1), or NaN: one where they
// are, else zero.
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
// The sum of values that are not finite: pos, neg: whether infinities of either
// sign are among them (NaN counts as both).
__device__ __forceinline__ float sum_of_marks(bool pos, bool neg) {
    return pos ? (neg ? __builtin_nanf("") : __builtin_inff()) : -__builtin_inff();
}

// Joins the parts of a split row group.  Every part wrote `rows` rows of sums
// [rows][D] and [rows] maxima and sums of weights with agent-scope stores, in
// slots `stride` floats apart from `part`.  `write(row, d, f32x4)` and
// `write_lse(row, value)` take the joined rows.  All threads of the workgroup
// take part; mx and den: LDS of `rows` floats each.
template <class T, int D, int Threads, class Row, class Lse>
__device__ __forceinline__ void join_parts(const float *part, int64_t stride, int n_parts, int rows,
                                           int row_slots, float *mx, float *den, Row write,
                                           Lse write_lse) {
    const int tid = threadIdx.x;
    for (int row = tid >> 4; row < rows; row += Threads / 16) {
        float m = kNoMax;
        for (int u = tid & 15; u < n_parts; u += 16)
            m = fmaxf(m, load_agent(part + u * stride + (int64_t)row_slots * D + row));
#pragma unroll
        for (int s = 8; s >= 1; s >>= 1) m = fmaxf(m, __shfl_xor(m, s));
        float l = 0.f;
        for (int u = tid & 15; u < n_parts; u += 16) {
            const float *p = part + u * stride + (int64_t)row_slots * D;
            l += load_agent(p + row_slots + row) * exp2_(load_agent(p + row) - m);
        }
#pragma unroll
        for (int s = 8; s >= 1; s >>= 1) l += __shfl_xor(l, s);
        if ((tid & 15) == 0) {
            mx[row] = m;
            den[row] = l;
            write_lse(row, l != 0.f ? (m + log2_(l) - T::kOff) * kLn2 : -__builtin_inff());
        }
    }
    __syncthreads();
    for (int i = tid; i < rows * (D / 4); i += Threads) {
        const int row = i / (D / 4), d = 4 * (i % (D / 4));
        const float m = mx[row], l = den[row];
        f32x4 sum = zero4();
        // Sixteen parts at a time, all of them on their way at once: one after
        // the other they cost most of a microsecond each.
        for (int u = 0; u < n_parts; u += 16) {
            f32x4 x[16];
            float f[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float *p = part + min(u + j, n_parts - 1) * stride;
                x[j] = __builtin_bit_cast(f32x4, buf_ld16<true>(buf_rsrc(p), 4u * (row * D + d)));
                f[j] = load_agent(p + (int64_t)row_slots * D + row);
            }
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (u + j < n_parts) sum += x[j] * part_factor(f[j] - m);
        }
        write(row, d, l != 0.f ? sum * (1.f / l) : zero4());
    }
}

}  // namespace serve
}  // namespace moe
