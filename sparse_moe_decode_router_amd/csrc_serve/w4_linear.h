// w4_linear.h - y = x W^T with 4-bit codes, a scale per group of 32, 64 or 128
// columns and, where there are any, zero points.
//
// Tokens are the rows and weight rows the columns of 16x16x32 MFMAs, so the
// scale and zero point of a weight row belong to one lane column and are
// applied to a group's sum in f32.  Codes become 16-bit floats without a
// conversion: bf16 0x4300 | q is 128 + q, fp16 0x6400 | q is 1024 + q, both
// exact, two at a time.  fp16 then subtracts 1024 + zero (exact, packed).
// bf16 has no packed subtraction: sum_j (128 + q_j) x_j - (128 + zero) sum_j
// x_j in f32, with the sums of x from one more MFMA against ones.  Partial sums
// are then up to 143 / 8 times larger than the result of a group, and lose that
// in f32: at most some 2^-18 of the sum of |x| scale, 2^-20 of the results as a
// whole, beside the output's own 2^-8.
// Pairs come out as (0,4)(1,5)(2,6)(3,7) of each eight codes, so x is put in
// that order.
//
// An operand load straight from memory would have neighbouring lanes in
// different rows, sixteen lines to a quarter of a wave: the texture addresser
// takes 64 cycles for such a load instead of 16, and was what bounded the
// kernel (9216 x 7168 codes, 8 tokens: 38 us).  So lanes load along the rows and
// the wave reorders through LDS (17 us; 15 with more rows per workgroup).
//
// What bounds it then: a single token with 36864 rows streams its codes at 3.9
// TB/s; with more tokens the vector unit, LDS and the addressers are each busy
// for about half of the time (8 tokens) and nothing alone stands out, with 64
// tokens x goes through LDS once per 32 weight rows.  More waves on a compute
// unit, or more steps ahead, measured no faster.
#pragma once

#include "serve_common.h"

namespace moe {
namespace serve {

struct W4Args {
    const uint16_t *x, *scales;
    const uint8_t *codes, *zeros;
    uint16_t *y;
    int64_t x_stride;
    int32_t tokens, k, n;
};

// Eight codes -> eight values in the order 0 4 1 5 2 6 3 7, without the zero.
// mask 0x000F000F and the magic are in registers, so that each pair of codes
// takes one and-or (two literals would not fit into one instruction).
__device__ __forceinline__ u32x4 w4_values(uint32_t c, uint32_t mask, uint32_t magic) {
    return (u32x4){(c & mask) | magic, (c >> 4 & mask) | magic, (c >> 8 & mask) | magic,
                   (c >> 12 & mask) | magic};
}
// Two packed halves minus two others.  (By value: a bit cast of a vector's
// element in place reads its first element.)
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, f16x2 b) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, a) - b);
}
__device__ __forceinline__ u32x4 w4_order(u32x4 x) {
    return (u32x4){__builtin_amdgcn_perm(x[2], x[0], 0x05040100u),
                   __builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
                   __builtin_amdgcn_perm(x[3], x[1], 0x05040100u),
                   __builtin_amdgcn_perm(x[3], x[1], 0x07060302u)};
}
// N bytes (1, 2, 4 or 8): from memory at any alignment, and to and from LDS at
// their own.
template <int N>
struct Packed {
    typedef uint64_t type;
};
template <>
struct Packed<4> {
    typedef uint32_t type;
};
template <>
struct Packed<2> {
    typedef uint16_t type;
};
template <>
struct Packed<1> {
    typedef uint8_t type;
};
template <int N>
__device__ __forceinline__ uint64_t ld_packed(const uint8_t *p) {
    typename Packed<N>::type v;
    __builtin_memcpy(&v, p, N);
    return v;
}
template <int N>
__device__ __forceinline__ uint64_t ld_aligned(const char *p) {
    return *(const typename Packed<N>::type *)p;
}
template <int N>
__device__ __forceinline__ void st_packed(char *p, uint64_t v) {
    *(typename Packed<N>::type *)p = (typename Packed<N>::type)v;
}

// One workgroup: 16 RT weight rows times 16 NT tokens; its W waves split K in
// steps of 128 columns, and every wave brings its own share of both operands:
// neighbouring lanes read neighbouring 16 bytes into registers, U steps ahead,
// and the wave turns them into operands through LDS of its own (no barrier).
// XR: x is brought by this many loads of four tokens each.  GL: log2 of the
// group; Z: zero points are given.
template <int NT, int XR, int RT, int W, int GL>
struct W4Lds {
    static constexpr int PG = 128 >> GL;        // groups of a step
    static constexpr int kX = 0, kCodes = XR * 1024, kScales = kCodes + RT * 1024;
    static constexpr int kZeros = kScales + RT * 128 * PG, kWave = kZeros + RT * 64 * PG;
    static constexpr int kSums = NT * RT * 1024;          // of one wave, in the end
    static constexpr int kBytes = W * (kWave > kSums ? kWave : kSums);
};
template <class T, int NT, int XR, int RT, int W, int U, int GL, bool Z>
__global__ __launch_bounds__(64 * W, NT * RT == 1 ? 4 : NT * RT < 16 ? 2 : 1) void k_w4(const W4Args a) {
    typedef W4Lds<NT, XR, RT, W, GL> Lds;
    constexpr bool kSums = T::kOne == 0x3F80u;  // bf16
    constexpr int PG = Lds::PG;
    __shared__ __attribute__((aligned(16))) char lds[Lds::kBytes];
    const int lane = lane_id(), wave = wave_index(), c = lane & 15, g = lane >> 4;
    const int n0 = (int)blockIdx.x * 16 * RT, t0 = (int)blockIdx.y * 16 * NT;
    const int groups = a.k >> GL, full = a.k >> 7;
    char *mine = lds + wave * Lds::kWave;

    // What a lane loads, as 32-bit offsets from the workgroup's first row: 16
    // bytes of x (row 4 i + lane / 16), 16 bytes of codes and a step's scales
    // (row lane / 4).
    const uint16_t *xb = a.x + t0 * a.x_stride;
    const uint8_t *codes = a.codes + (int64_t)n0 * (a.k / 2);
    const uint8_t *scales = (const uint8_t *)(a.scales + (int64_t)n0 * groups);
    const uint8_t *zeros = Z ? a.zeros + (int64_t)n0 * groups : nullptr;
    uint32_t xo[XR], co[RT], go[RT];
#pragma unroll
    for (int i = 0; i < XR; ++i)
        xo[i] = 2 * (uint32_t)min(4 * i + g, a.tokens - 1 - t0) * (uint32_t)a.x_stride + 16 * c;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const uint32_t row = min(16 * r + (lane >> 2), a.n - 1 - n0);
        co[r] = row * (a.k / 2) + 16 * (lane & 3);
        go[r] = row * groups;
    }
    // Where it puts them, and where operands are read.  Codes: of a row's 64
    // bytes, dword 4 i + j of memory (columns 32 i + 8 j ..) goes to 4 j + i, so
    // that lane group g finds its columns of the four MFMA steps in one piece;
    // both there and in x pieces of 16 bytes change places within a row, for
    // the sake of the banks.
    uint32_t codes_w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        codes_w[j] = Lds::kCodes + (lane >> 2) * 64 + 16 * (j ^ (lane >> 4)) + 4 * (lane & 3);
    const uint32_t codes_r = Lds::kCodes + c * 64 + 16 * (g ^ (c >> 2));
    constexpr int kRows = 4 * XR < 16 ? 4 * XR : 16;   // of a tile of x that are there
    const int xc = c & (kRows - 1);

    f32x4 acc[NT][RT], part[NT][RT], sums[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        sums[t] = zero4();
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[t][r] = part[t][r] = zero4();
    }
    constexpr uint32_t one2 = T::kOne | T::kOne << 16;
    const u32x4 ones = {one2, one2, one2, one2};
    uint32_t mask = 0x000F000Fu, magic = kSums ? 0x43004300u : 0x64006400u;
    asm("" : "+v"(mask), "+v"(magic));

    struct Step {
        u32x4 code[RT], x[XR];
    } ring[U];
    struct Scales {
        uint64_t scale[RT];
        uint32_t zero[RT];
    };
    auto load = [&](Step &d, int s) {
#pragma unroll
        for (int r = 0; r < RT; ++r) d.code[r] = ld_weight16(codes + 64 * s + co[r]);
#pragma unroll
        for (int i = 0; i < XR; ++i) d.x[i] = ld16((const char *)xb + 256 * s + xo[i]);
    };
    auto put = [&](const Step &d) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *(uint32_t *)(mine + codes_w[j] + 1024 * r) = d.code[r][j];
#pragma unroll
        for (int i = 0; i < XR; ++i) {
            const int row = 4 * i + g;
            *(u32x4 *)(mine + Lds::kX + row * 256 + 16 * (c ^ (row & 15))) = w4_order(d.x[i]);
        }
    };
    // Scales and zero points come for four steps at a time, one per lane.
    auto load_scales = [&](Scales &d, int s, int last) {
        const uint32_t at = PG * min(s + (lane & 3), last);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            d.scale[r] = ld_packed<2 * PG>(scales + 2 * (go[r] + at));
            d.zero[r] = Z ? (uint32_t)ld_packed<PG>(zeros + (go[r] + at)) : 0u;
        }
    };
    auto put_scales = [&](const Scales &d) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            st_packed<2 * PG>(mine + Lds::kScales + 2 * PG * (64 * r + lane), d.scale[r]);
            if constexpr (Z) st_packed<PG>(mine + Lds::kZeros + PG * (64 * r + lane), d.zero[r]);
        }
    };
    // The step in LDS; u: its place among four.
    auto multiply = [&](int u) {
        u32x4 code[RT];
        uint64_t sc[RT];
        uint32_t zr[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int at = 64 * r + 4 * c + u;
            code[r] = ld16(mine + codes_r + 1024 * r);
            sc[r] = ld_aligned<2 * PG>(mine + Lds::kScales + 2 * PG * at);
            zr[r] = Z ? (uint32_t)ld_aligned<PG>(mine + Lds::kZeros + PG * at) : 0u;
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int gi = 32 * m >> GL;
            u32x4 x[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t)
                x[t] = ld16(mine + Lds::kX + (16 * t + xc) * 256 + 16 * ((4 * m + g) ^ xc));
            if constexpr (kSums) {
#pragma unroll
                for (int t = 0; t < NT; ++t) sums[t] = T::mfma16(x[t], ones, sums[t]);
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const uint32_t z = Z ? zr[r] >> 8 * gi & 255u : 8u;
                u32x4 w = w4_values(code[r][m], mask, magic);
                if constexpr (!kSums) {
                    // fp16 of 1024 + z, twice
                    const f16x2 z2 = __builtin_bit_cast(f16x2, 0x64006400u | z | z << 16);
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = sub_f16x2(w[i], z2);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) part[t][r] = T::mfma16(x[t], w, part[t][r]);
            }
            if ((32 * (m + 1) & ((1 << GL) - 1)) == 0) {
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const float scale = T::lo((uint32_t)(sc[r] >> 16 * gi));
                    const float z = 128.f + (Z ? (float)(zr[r] >> 8 * gi & 255u) : 8.f);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float p = kSums ? fmaf(-z, sums[t][i], part[t][r][i])
                                                  : part[t][r][i];
                            acc[t][r][i] = fmaf(scale, p, acc[t][r][i]);
                        }
                        part[t][r] = zero4();
                    }
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) sums[t] = zero4();
            }
        }
    };

    const int s0 = (int)((int64_t)full * wave / W), s1 = (int)((int64_t)full * (wave + 1) / W);
    if (s0 < s1) {
        Scales sc;
        load_scales(sc, s0, s1 - 1);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // In this order, so that the loop waits for the oldest alone.
            __builtin_amdgcn_sched_barrier(0);
            load(ring[u], min(s0 + u, s1 - 1));
        }
        __builtin_amdgcn_sched_barrier(0);
        for (int s = s0; s < s1; s += U) {
            if (((s - s0) & 3) == 0) {
                put_scales(sc);
                load_scales(sc, s + 4, s1 - 1);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (s + u >= s1) break;
                put(ring[u]);
                load(ring[u], min(s + u + U, s1 - 1));
                wave_sync();
                multiply((s + u - s0) & 3);
                wave_sync();
            }
        }
    }
    if (wave == W - 1 && (a.k & 127)) {
        // What is left of K, up to three blocks of 32 columns: what is not
        // there is zero.
        Step d;
        Scales sc;
        const int left = a.k & 127, n_groups = left >> GL;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            d.code[r] = (u32x4){0, 0, 0, 0};
            if (32 * (lane & 3) < left) d.code[r] = ld_weight16(codes + (co[r] + 64 * full));
            sc.scale[r] = 0;
            sc.zero[r] = 0;
#pragma unroll
            for (int i = 0; i < PG; ++i) {
                if (i >= n_groups) break;
                const uint32_t at = go[r] + PG * full + i;
                sc.scale[r] |= (uint64_t)*(const uint16_t *)(scales + 2 * at) << 16 * i;
                if constexpr (Z) sc.zero[r] |= (uint32_t)zeros[at] << 8 * i;
            }
        }
#pragma unroll
        for (int i = 0; i < XR; ++i) {
            d.x[i] = (u32x4){0, 0, 0, 0};
            if (8 * c < left) d.x[i] = ld16((const char *)xb + (xo[i] + 256 * full));
        }
        put(d);
        put_scales(sc);
        wave_sync();
        multiply(0);
    }
    __syncthreads();  // the same memory now takes the waves' sums
    f32x4 *s_acc = (f32x4 *)lds;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < RT; ++r) s_acc[(wave * NT * RT + t * RT + r) * 64 + lane] = acc[t][r];
    __syncthreads();
    // Element (tile, token i of lane group, column): summed in wave order.
    for (int i = threadIdx.x; i < NT * RT * 64; i += 64 * W) {
        const int l = i & 63, tr = i >> 6, t = tr / RT, r = tr % RT;
        f32x4 sum = zero4();
#pragma unroll
        for (int w = 0; w < W; ++w) sum += s_acc[(w * NT * RT + tr) * 64 + l];
        const int col = n0 + 16 * r + (l & 15);
        if (col >= a.n) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int tok = t0 + 16 * t + 4 * (l >> 4) + e;
            if (tok < a.tokens) a.y[(int64_t)tok * a.n + col] = (uint16_t)T::pack(sum[e], 0.f);
        }
    }
}

}  // namespace serve
}  // namespace moe
