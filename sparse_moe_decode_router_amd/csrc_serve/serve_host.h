// serve_host.h - what the host sides of the serving operators share: status of
// launches, the device's compute units, checks of arguments and the choice of a
// kernel by types and head_dim.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "moe_serve.h"
#include "serve_common.h"

namespace moe {
namespace serve {

inline thread_local int32_t g_last_hip = 0;

inline moe_status hip_error(hipError_t e) {
    g_last_hip = (int32_t)e;
    return MOE_ERR_HIP;
}
inline moe_status launched() {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? MOE_OK : hip_error(e);
}

// Compute units of the current device (0: unknown yet, -1: not gfx950).
constexpr int kMaxDevices = 64;
inline std::atomic<int> g_cus[kMaxDevices];

inline moe_status compute_units(int *cus) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_error(e);
    if (dev < 0 || dev >= kMaxDevices) return MOE_ERR_UNSUPPORTED;
    int n = g_cus[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        hipDeviceProp_t p;
        e = hipGetDeviceProperties(&p, dev);
        if (e != hipSuccess) return hip_error(e);
        const bool ours = p.gcnArchName[0] == 'g' && std::equal(p.gcnArchName, p.gcnArchName + 6, "gfx950");
        n = ours ? p.multiProcessorCount : -1;
        g_cus[dev].store(n, std::memory_order_relaxed);
    }
    if (n < 0) return MOE_ERR_UNSUPPORTED;
    *cus = n;
    return MOE_OK;
}

inline bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
inline int log2_of(int v) {
    int r = 0;
    while ((1 << r) < v) ++r;
    return r;
}
inline int64_t plane_bytes(const moe_kv_cache &kv) {
    return (int64_t)kv.pages * kv.kv_heads * kv.page * kv.head_dim * (kv.dtype == MOE_E4M3 ? 1 : 2);
}
inline char *plane(const moe_kv_cache &kv, int layer, int which) {
    return (char *)kv.data + (2 * (int64_t)layer + which) * plane_bytes(kv);
}

constexpr int kMaxRows = 1 << 24;  // sequences, tokens of a call, pairs of a list
// A grid's first axis has below 2^32 threads, its second up to 2^16 workgroups.
constexpr int64_t kMaxGrid256 = (1ll << 24) - 1;   // of 256 threads each

// Workgroups that one decode call aims at: with four waves each, three of them
// share a compute unit.
constexpr int kUnitsPerCu = 4;
// What a plan is made for; the device a plan runs on has the same number.
constexpr int kPlanCus = 256;

// keys: of the longest sequence.
inline int decode_split(const moe_kv_cache &kv, const moe_attn_config &c, int64_t keys) {
    const int group = c.q_heads / kv.kv_heads, hg = (group + 15) / 16;
    const int heads = kv.kv_heads * hg;
    // No unit is smaller than a block per wave.
    if (c.window > 0) keys = std::min<int64_t>(keys, (int64_t)c.window + c.sinks + 62);
    const int64_t most = (int64_t)c.batch * ((keys + 127) / 128);
    return (int)std::max<int64_t>(
        1, std::min<int64_t>(most, std::max(1, kPlanCus * kUnitsPerCu / heads)));
}

// Workgroups of a prompt call that the chip holds at once.
inline int prompt_slots(int head_dim) { return kPlanCus * (head_dim <= 128 ? 2 : 1); }

template <class F>
moe_status with_dim(int d, F f) {
    switch (d) {
        case 64: return f(std::integral_constant<int, 64>());
        case 96: return f(std::integral_constant<int, 96>());
        case 128: return f(std::integral_constant<int, 128>());
        case 192: return f(std::integral_constant<int, 192>());
        case 256: return f(std::integral_constant<int, 256>());
    }
    return MOE_ERR_UNSUPPORTED;
}
// Calls f with the compute type and whether the cache holds e4m3.
template <class F>
moe_status with_types(int dtype, bool f8, F f) {
    if (dtype == MOE_BF16) return f8 ? f(Bf16(), std::true_type()) : f(Bf16(), std::false_type());
    return f8 ? f(Fp16(), std::true_type()) : f(Fp16(), std::false_type());
}

inline moe_status check_types(const moe_kv_cache &kv, int dtype) {
    if (dtype != MOE_BF16 && dtype != MOE_FP16) return MOE_ERR_INVALID_ARG;
    if (kv.dtype != MOE_E4M3 && kv.dtype != dtype) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}
inline moe_status check_strides(int64_t token, int64_t head, int heads, int d) {
    if (token < 0 || head < 0 || (token | head) % 8) return MOE_ERR_INVALID_ARG;
    if (heads > 1 && head < d) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

inline AttnArgs attn_args(const moe_kv_cache &kv, const moe_attn_config &c, int layer) {
    AttnArgs a = {};
    a.k = plane(kv, layer, 0);
    a.v = plane(kv, layer, 1);
    a.tables = kv.tables;
    a.lengths = kv.lengths;
    a.k_scale = kv.k_scale;
    a.v_scale = kv.v_scale;
    a.scale = c.scale * moe::serve::kLog2e;
    a.pages = kv.pages;
    a.cols = kv.cols;
    a.page_log2 = log2_of(kv.page);
    a.kv_heads = kv.kv_heads;
    a.group = c.q_heads / kv.kv_heads;
    a.head_groups = (a.group + 15) / 16;
    a.window = c.window;
    a.sinks = c.window > 0 ? c.sinks : 0;
    return a;
}

inline moe_status check_attn(const moe_kv_cache *kv, const moe_attn_config *c, int layer, const void *q,
                      int dtype, int64_t token, int64_t head, int batch, const void *out,
                      const void *lse, const void *ws, const void *counters) {
    moe_status s = moe_attn_validate(kv, c);
    if (s != MOE_OK) return s;
    if (!q || !out || !lse || batch < 1 || batch > c->batch || layer < 0 || layer >= kv->layers)
        return MOE_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4)) return MOE_ERR_INVALID_ARG;
    if ((s = check_types(*kv, dtype)) != MOE_OK) return s;
    if ((s = check_strides(token, head, c->q_heads, kv->head_dim)) != MOE_OK) return s;
    if (!aligned(ws, 16) || !aligned(counters, 16)) return MOE_ERR_WORKSPACE;
    return MOE_OK;
}

}  // namespace serve
}  // namespace moe
