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
    uint32_t T;                 // 0: everything is kept and nothing below is read
    uint32_t last;              // 65536 T - 1: a draw in a word's high half is dropped up to here
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
    // x of column e (of the eight) after dropout; a dropped NaN or infinity
    // is 0.  (A draw u in the high half and anything below it: u < T where
    // the word is at most 65536 T - 1, so the odd columns need no shift.)
    __device__ __forceinline__ float apply(float x, const uint32_t (&w)[4], int e) const { return mask(x * scale, w, e); }
    __device__ __forceinline__ float mask(float x, const uint32_t (&w)[4], int e) const {
        const uint32_t u = (e & 1) ? w[e / 2] : w[e / 2] << 16;
        return u > last ? x : 0.f;
    }
};

// Checks a caller's sag_drop (null: no dropout) for `rows` rows.
inline sag_status make_drop(const char* who, const sag_drop* d, int64_t rows, DropArgs* out) {
    *out = DropArgs{};
    if (!d) return SAG_OK;
    if (!(d->p >= 0.f && d->p <= 1.f)) return fail(SAG_E_INVALID, std::string(who) + ": dropout p outside [0, 1]");
    const uint32_t T = static_cast<uint32_t>(std::floor(static_cast<double>(d->p) * 65536.0 + 0.5));
    if (T == 0) return SAG_OK;
    if (!d->nodes && (d->row0 < 0 || d->row0 > (int64_t{1} << 32) - rows))
        return fail(SAG_E_INVALID, std::string(who) + ": dropout row ids outside 32 bits");
    out->T = T;
    out->last = (T << 16) - 1u;   // T = 65536: all ones
    out->scale = T == 65536u ? 0.f : static_cast<float>(65536.0 / (65536.0 - T));
    out->key0 = static_cast<uint32_t>(d->seed);
    out->key1 = static_cast<uint32_t>(d->seed >> 32);
    out->call = d->call;
    out->row0 = d->nodes ? 0u : static_cast<uint32_t>(d->row0);
    out->call_dev = d->call_dev;
    out->nodes = d->nodes;
    return SAG_OK;
}

// Two fp32 values as packed bf16 (round to nearest even, one instruction).
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    const f32x2_t v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

// Stores the first n (1 to V) of a vector's worth of values at p, 16-byte
// aligned; written out so that the values stay in registers.
template <class T>
__device__ __forceinline__ void store_first(T* p, const float* f, int n) {
    constexpr int V = Vec<T>::N;
    if (n >= V) {
        if constexpr (V == 8)
            *reinterpret_cast<uint4*>(p) = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
        else
            *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < n) p[e] = from_f32<T>(f[e]);
    }
}

inline bool act_ok(sag_act a) { return a >= SAG_ACT_NONE && a <= SAG_ACT_SILU; }

// The tail of the normal distribution: for a = |z|
//   1 - Phi(a) = exp(-a^2 / 2) t P(t),  t = 1 / (1 + c a),
// where t P(t) stands for half the scaled complementary error function.  P is
// a least-maximum fit on [0, 14], beyond which the exponential is 0 in fp32
// (Lawson's reweighted least squares on 12,000 points): of relative error
// 1.5e-7 with eight terms and c = 0.3 (FINE: fp32 results and gradients), of
// 3.1e-5 with five and c = 0.375 (values that are then rounded to bf16, half a
// step of which is 3.9e-3).  The tail keeps its relative accuracy, and the
// exponential, e = exp(-a^2 / 2), is also the density that the derivative
// needs.  The library's erfcf, which branches by range, took 1.3 ms against
// 0.9 ms for this in the gradient pass over 2.45M x 256 bf16 (5.0 GB).
template <bool FINE>
__device__ __forceinline__ float normal_tail(float z, float& e) {
    const float t = __builtin_amdgcn_rcpf(fmaf(FINE ? 0.3f : 0.375f, fabsf(z), 1.f));
    e = __builtin_amdgcn_exp2f(z * z * -0.72134752044448170f);   // exp(-z^2 / 2)
    float p;
    if constexpr (FINE) {
        p = fmaf(0.0356758525f, t, -0.157207547f);
        p = fmaf(p, t, 0.206361131f);
        p = fmaf(p, t, -0.0536906036f);
        p = fmaf(p, t, 0.128565293f);
        p = fmaf(p, t, 0.0999123772f);
        p = fmaf(p, t, 0.120754137f);
        p = fmaf(p, t, 0.119629287f);
    } else {
        p = fmaf(-0.0906485941f, t, 0.200294511f);
        p = fmaf(p, t, 0.0835541374f);
        p = fmaf(p, t, 0.157737088f);
        p = fmaf(p, t, 0.149060699f);
    }
    return p * t * e;
}

__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
}

// act(z) in fp32, for a result of type T.  ReLU keeps NaN.
template <int ACT, class T>
__device__ __forceinline__ float act_value(float z, float slope) {
    if constexpr (ACT == SAG_ACT_RELU) return z < 0.f ? 0.f : z;
    else if constexpr (ACT == SAG_ACT_LEAKY_RELU) return z > 0.f ? z : z * slope;
    else if constexpr (ACT == SAG_ACT_GELU) {
        // z Phi(z) = max(z, 0) - |z| (1 - Phi(|z|))
        float e;
        const float q = normal_tail<sizeof(T) == 4>(z, e);
        return fmaf(-fminf(fabsf(z), 32.f), q, z < 0.f ? 0.f : z);   // (q is 0 there, and infinity stays)
    } else if constexpr (ACT == SAG_ACT_SILU) return z * sigmoid(z);
    else return z;
}

// act'(z): 0 at z = 0 for ReLU, `slope` there for leaky ReLU.
template <int ACT>
__device__ __forceinline__ float act_grad(float z, float slope) {
    if constexpr (ACT == SAG_ACT_RELU) return z > 0.f ? 1.f : 0.f;
    else if constexpr (ACT == SAG_ACT_LEAKY_RELU) return z > 0.f ? 1.f : slope;
    else if constexpr (ACT == SAG_ACT_GELU) {
        float e;
        const float q = normal_tail<true>(z, e);
        return fmaf(z * 0.39894228040143268f, e, z < 0.f ? q : 1.f - q);   // Phi + z phi
    } else if constexpr (ACT == SAG_ACT_SILU) {
        const float s = sigmoid(z);
        return s * fmaf(z, 1.f - s, 1.f);
    } else return 1.f;
}

// g act'(z); where ReLU is off the result is 0 whatever g is.
template <int ACT>
__device__ __forceinline__ float times_act_grad(float g, float z, float slope) {
    if constexpr (ACT == SAG_ACT_RELU) return z > 0.f ? g : 0.f;
    else return g * act_grad<ACT>(z, slope);
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
