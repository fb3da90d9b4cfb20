// Dropout masks and activations as the kernels use them.
//
// The mask is a function of (seed, call, node, column) and is never stored:
// element j of the row with stream id `node` is kept when its 16-bit draw,
// number j % 8 of the Philox4x32-10 block at counter (j / 8, node, call, 1),
// is at least T = round(65536 p).  Sixteen bits a draw make one block serve
// the eight elements of a 16-byte bf16 vector (at four draws a block the
// generator, not HBM, would set the rate of a bf16 pass: 20 quarter-rate
// multiplies a block against 32 bytes of traffic); p is taken to the nearest
// 2^-16 and the kept values are scaled by 65536 / (65536 - T), so the
// expectation is exact for the p that is used.
#pragma once

#include <cmath>

#include "philox.h"

namespace sag {

struct DropArgs {
    uint32_t T;                 // 0: everything is kept
    float scale;                // 65536 / (65536 - T); 0 when T = 65536
    uint32_t key0, key1, call, row0;
    const uint32_t* call_dev;   // nullable: added to call when the kernel runs
    const int32_t* nodes;       // nullable: stream id of each row

    __device__ __forceinline__ uint32_t call_now() const { return call + (call_dev ? *call_dev : 0u); }
    __device__ __forceinline__ uint32_t node_of(int64_t row) const {
        return nodes ? static_cast<uint32_t>(nodes[row]) : row0 + static_cast<uint32_t>(row);
    }
    // The eight draws of columns 8 g .. 8 g + 7 (two per word, low half first).
    __device__ __forceinline__ void draws(uint32_t node, uint32_t g, uint32_t call_word, uint32_t (&w)[4]) const {
        w[0] = g;
        w[1] = node;
        w[2] = call_word;
        w[3] = 1u;
        philox4x32_10(w, key0, key1);
    }
    // x of column e (of the eight) after dropout; a dropped NaN or infinity is 0.
    __device__ __forceinline__ float apply(float x, const uint32_t (&w)[4], int e) const {
        const uint32_t u = (e & 1) ? w[e / 2] >> 16 : w[e / 2] & 0xffffu;
        return u >= T ? x * scale : 0.f;
    }
};

// Checks a caller's sag_drop (null: no dropout) for `rows` rows.
inline sag_status make_drop(const char* who, const sag_drop* d, int64_t rows, DropArgs* out) {
    *out = DropArgs{0u, 1.f, 0u, 0u, 0u, 0u, nullptr, nullptr};
    if (!d) return SAG_OK;
    if (!(d->p >= 0.f && d->p <= 1.f)) return fail(SAG_E_INVALID, std::string(who) + ": dropout p outside [0, 1]");
    const uint32_t T = static_cast<uint32_t>(std::floor(static_cast<double>(d->p) * 65536.0 + 0.5));
    if (T == 0) return SAG_OK;
    if (!d->nodes && (d->row0 < 0 || d->row0 > (int64_t{1} << 32) - rows))
        return fail(SAG_E_INVALID, std::string(who) + ": dropout row ids outside 32 bits");
    out->T = T;
    out->scale = T == 65536u ? 0.f : static_cast<float>(65536.0 / (65536.0 - T));
    out->key0 = static_cast<uint32_t>(d->seed);
    out->key1 = static_cast<uint32_t>(d->seed >> 32);
    out->call = d->call;
    out->row0 = d->nodes ? 0u : static_cast<uint32_t>(d->row0);
    out->call_dev = d->call_dev;
    out->nodes = d->nodes;
    return SAG_OK;
}

inline bool act_ok(sag_act a) { return a >= SAG_ACT_NONE && a <= SAG_ACT_SILU; }

constexpr float kSqrtHalf = 0.70710678118654752f, kInvSqrt2Pi = 0.39894228040143268f;

// act(z) in fp32.  ReLU keeps NaN; GELU is z times the normal distribution
// function, through erfc so that the left tail keeps its relative accuracy.
template <int ACT>
__device__ __forceinline__ float act_value(float z, float slope) {
    if constexpr (ACT == SAG_ACT_RELU) return z < 0.f ? 0.f : z;
    else if constexpr (ACT == SAG_ACT_LEAKY_RELU) return z > 0.f ? z : z * slope;
    else if constexpr (ACT == SAG_ACT_GELU) return 0.5f * z * erfcf(-kSqrtHalf * z);
    else if constexpr (ACT == SAG_ACT_SILU) return z / (1.f + expf(-z));
    else return z;
}

// act'(z): 0 at z = 0 for ReLU, `slope` there for leaky ReLU.
template <int ACT>
__device__ __forceinline__ float act_grad(float z, float slope) {
    if constexpr (ACT == SAG_ACT_RELU) return z > 0.f ? 1.f : 0.f;
    else if constexpr (ACT == SAG_ACT_LEAKY_RELU) return z > 0.f ? 1.f : slope;
    else if constexpr (ACT == SAG_ACT_GELU)
        return 0.5f * erfcf(-kSqrtHalf * z) + z * (kInvSqrt2Pi * expf(-0.5f * z * z));
    else if constexpr (ACT == SAG_ACT_SILU) {
        const float e = 1.f / (1.f + expf(-z));
        return e * (1.f + z * (1.f - e));
    } else return 1.f;
}

// f(std::integral_constant<int, act>) for a runtime activation.
template <class F>
auto with_act(sag_act a, F&& f) {
    switch (a) {
        case SAG_ACT_RELU: return f(std::integral_constant<int, SAG_ACT_RELU>{});
        case SAG_ACT_LEAKY_RELU: return f(std::integral_constant<int, SAG_ACT_LEAKY_RELU>{});
        case SAG_ACT_GELU: return f(std::integral_constant<int, SAG_ACT_GELU>{});
        case SAG_ACT_SILU: return f(std::integral_constant<int, SAG_ACT_SILU>{});
        default: return f(std::integral_constant<int, SAG_ACT_NONE>{});
    }
}

}  // namespace sag
