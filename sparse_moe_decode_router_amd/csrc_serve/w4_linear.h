// w4_linear.h - y = x W^T with 4-bit codes, a scale per group of 32, 64 or 128
// columns and, where there are any, zero points.
//
// Tokens are the rows and weight rows the columns of 16x16x32 MFMAs, so the
// scale and zero point of a weight row belong to one lane column and are
// applied to a group's sum in f32.  A lane reads 16 bytes of a row (32 codes;
// its four lane groups read 128 consecutive columns), a 4x4 exchange of dwords
// among the lane groups gives MFMA m the columns 32m .. 32m + 31, eight
// consecutive ones per lane group.  Codes become 16-bit floats without a
// conversion: bf16 0x4300 | q is 128 + q, fp16 0x6400 | q is 1024 + q, both
// exact, two at a time.  fp16 then subtracts 1024 + zero (exact, packed).
// bf16 has no packed subtraction: sum_j (128 + q_j) x_j - (128 + zero) sum_j
// x_j in f32, with the sums of x from one more MFMA against ones.
// Pairs come out as (0,4)(1,5)(2,6)(3,7) of each eight codes, so x is put in
// that order.
#pragma once

#include "serve_common.h"

namespace moe {
namespace serve {

struct W4Args {
    const uint16_t *x, *scales;
    const uint8_t *codes, *zeros;
    uint16_t *y;
    float *part;
    uint32_t *counters;
    int64_t x_stride;
    int32_t tokens, k, n, group_log2;
    int32_t steps, slices;       // K in steps of 128, split over this many workgroups
};

constexpr int kW4Waves = 8;
constexpr int kW4Threads = 64 * kW4Waves;

// Eight codes -> eight values in the order 0 4 1 5 2 6 3 7, without the zero.
template <class T>
__device__ __forceinline__ u32x4 w4_values(uint32_t c) {
    constexpr uint32_t kMagic = T::kOne == 0x3F80u ? 0x43004300u : 0x64006400u;
    return (u32x4){(c & 0x000F000Fu) | kMagic, (c >> 4 & 0x000F000Fu) | kMagic,
                   (c >> 8 & 0x000F000Fu) | kMagic, (c >> 12 & 0x000F000Fu) | kMagic};
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
__device__ __forceinline__ u32x4 w4_exchange(u32x4 c) {
    const auto a = __builtin_amdgcn_permlane32_swap(c[0], c[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(c[1], c[3], false, false);
    const auto p = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto q = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return (u32x4){p[0], p[1], q[0], q[1]};
}

// One workgroup: 16 RT weight rows, NT tiles of 16 tokens; its waves split K.
template <class T, int NT, int RT>
__global__ __launch_bounds__(kW4Threads) void k_w4(const W4Args a) {
    constexpr bool kSums = T::kOne == 0x3F80u;  // bf16
    __shared__ f32x4 s_acc[kW4Waves][NT * RT][64];
    const int lane = lane_id(), wave = wave_index(), c = lane & 15, g = lane >> 4;
    const int n0 = (int)blockIdx.x * 16 * RT, t0 = (int)blockIdx.y * 16 * NT;

    const uint8_t *cp[RT];
    const uint16_t *sp[RT];
    const uint8_t *zp[RT];
    const int groups = a.k >> a.group_log2;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int64_t row = min(n0 + 16 * r + c, a.n - 1);
        cp[r] = a.codes + row * (a.k / 2) + 16 * g;
        sp[r] = a.scales + row * groups;
        zp[r] = a.zeros ? a.zeros + row * groups : nullptr;
    }
    const uint16_t *xp[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
        xp[t] = a.x + min(t0 + 16 * t + c, a.tokens - 1) * a.x_stride + 8 * g;

    f32x4 acc[NT][RT], part[NT][RT], sums[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        sums[t] = zero4();
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[t][r] = part[t][r] = zero4();
    }
    constexpr uint32_t one2 = T::kOne | T::kOne << 16;
    const u32x4 ones = {one2, one2, one2, one2};
    const int per_group = 1 << (a.group_log2 - 5);  // MFMA steps of 32 columns

    const int steps = a.steps;
    const int s0 = (int)((int64_t)steps * wave / kW4Waves),
              s1 = (int)((int64_t)steps * (wave + 1) / kW4Waves);
    // One step of 128 columns, or what is left of them.
    auto multiply = [&](u32x4 *code, int s) {
#pragma unroll
        for (int r = 0; r < RT; ++r) code[r] = w4_exchange(code[r]);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int k = 128 * s + 32 * m;
            if (k >= a.k) continue;
            const int gi = k >> a.group_log2;
            u32x4 x[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) x[t] = w4_order(ld16(xp[t] + k));
            if constexpr (kSums) {
#pragma unroll
                for (int t = 0; t < NT; ++t) sums[t] = T::mfma16(x[t], ones, sums[t]);
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                u32x4 w = w4_values<T>(code[r][m]);
                if constexpr (!kSums) {
                    const uint32_t z = 1024u + (a.zeros ? zp[r][gi] : 8u);
                    const _Float16 zh = (_Float16)(float)z;
                    const f16x2 z2 = {zh, zh};
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = sub_f16x2(w[i], z2);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) part[t][r] = T::mfma16(x[t], w, part[t][r]);
            }
            if (((k >> 5) + 1) % per_group == 0) {
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const float scale = T::lo(sp[r][gi]);
                    const float z = 128.f + (a.zeros ? (float)zp[r][gi] : 8.f);
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
    for (int s = s0; s < s1; ++s) {
        u32x4 code[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            code[r] = (u32x4){0, 0, 0, 0};
            if (128 * s + 32 * g < a.k) code[r] = ld_weight16(cp[r] + 64 * s);
        }
        multiply(code, s);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < RT; ++r) s_acc[wave][t * RT + r][lane] = acc[t][r];
    __syncthreads();
    // Element (tile, token i of lane group, column): summed in wave order.
    for (int x = threadIdx.x; x < NT * RT * 64; x += kW4Threads) {
        const int l = x & 63, tr = x >> 6, t = tr / RT, r = tr % RT;
        f32x4 sum = zero4();
#pragma unroll
        for (int w = 0; w < kW4Waves; ++w) sum += s_acc[w][tr][l];
        const int col = n0 + 16 * r + (l & 15);
        if (col >= a.n) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int tok = t0 + 16 * t + 4 * (l >> 4) + i;
            if (tok < a.tokens) a.y[(int64_t)tok * a.n + col] = (uint16_t)T::pack(sum[i], 0.f);
        }
    }
}

}  // namespace serve
}  // namespace moe
