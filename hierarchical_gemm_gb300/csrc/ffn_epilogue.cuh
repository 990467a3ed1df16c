// ffn_epilogue.cuh -- what the feed-forward operators do with an fp32
// accumulator before it is stored: the bias, the activations (and their
// derivatives, for the backward pass), the residual and the saved
// pre-activations.
//
// Everything here is fp32 on sums the tensor cores made in fp32; the one
// rounding to 16 bits is the store's.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>
#include <type_traits>

#include "ffn_kernels.h"
#include "ptx.cuh"

namespace tsg {

// The activations (the tsffn_act_t values).
enum ActKind { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4, kActSigmoid = 5 };

// 1 / (1 + 2^-t), within a few fp32 ulps (ex2.approx, a fast division).
// t -> -inf gives 1 / inf = 0, t -> inf gives 1.
__device__ __forceinline__ float sigmoid_log2(float t) { return __fdividef(1.0f, 1.0f + ex2_approx(-t)); }

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTanhCubic = 0.044715f;                 // the tanh form's cubic coefficient
constexpr float kTanhScale = 1.5957691216057308f;       // 2 sqrt(2 / pi)
constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

// The tanh form of gelu is z sigma(2 sqrt(2 / pi) (z + 0.044715 z^3)), since
// (1 + tanh u) / 2 = sigma(2 u): one exponential, no cancellation for z < 0.
__device__ __forceinline__ float gelu_tanh_gate(float z) {
    return sigmoid_log2(kTanhScale * kLog2e * z * fmaf(kTanhCubic * z, z, 1.0f));
}
// gelu is z Phi(z) with Phi(z) = erfc(-z / sqrt 2) / 2, which keeps its
// relative accuracy in the tail where 1 + erf cancels.
__device__ __forceinline__ float normal_cdf(float z) { return 0.5f * erfcf(-kSqrtHalf * z); }

template <int kAct>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (kAct == kActRelu) return z < 0.0f ? 0.0f : z;  // (a NaN stays one)
    if constexpr (kAct == kActGelu) return z * normal_cdf(z);
    if constexpr (kAct == kActGeluTanh) return z * gelu_tanh_gate(z);
    if constexpr (kAct == kActSilu) return z * sigmoid_log2(kLog2e * z);
    if constexpr (kAct == kActSigmoid) return sigmoid_log2(kLog2e * z);
    return z;
}

// act(z) and act'(z).
template <int kAct>
__device__ __forceinline__ void act_both(float z, float& a, float& da) {
    if constexpr (kAct == kActRelu) {
        a = z < 0.0f ? 0.0f : z;
        da = z > 0.0f ? 1.0f : 0.0f;
    } else if constexpr (kAct == kActGelu) {
        const float p = normal_cdf(z);
        a = z * p;
        da = fmaf(z * kInvSqrt2Pi, ex2_approx(-0.5f * kLog2e * z * z), p);
    } else if constexpr (kAct == kActGeluTanh) {
        const float s = gelu_tanh_gate(z);
        a = z * s;
        // s (1 - s) is exactly 0 well before |z| = 16; the clamp keeps z^2
        // finite for the largest z, where 0 * inf would be NaN
        const float c = fminf(fmaxf(z, -16.0f), 16.0f);
        da = fmaf(c * s * (1.0f - s), kTanhScale * fmaf(3.0f * kTanhCubic * c, c, 1.0f), s);
    } else if constexpr (kAct == kActSilu) {
        const float s = sigmoid_log2(kLog2e * z);
        a = z * s;
        da = s * fmaf(z, 1.0f - s, 1.0f);
    } else if constexpr (kAct == kActSigmoid) {
        a = sigmoid_log2(kLog2e * z);
        da = a * (1.0f - a);
    } else {
        a = z;
        da = 1.0f;
    }
}

// f(z) is called with the activation as a compile-time value.
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
    switch (act) {
        case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
        case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
        case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>{}); break;
        case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
        case kActSigmoid: f(std::integral_constant<int, kActSigmoid>{}); break;
        default: f(std::integral_constant<int, kActNone>{}); break;
    }
}

// ------------------------------------------------- 16-bit / fp32 vectors --

// The two 16-bit floats of a word (the low half is the lower index).
template <bool kBF16>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
    if constexpr (kBF16) {
        return {__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)};
    } else {
        __half2 h;
        memcpy(&h, &w, 4);
        return __half22float2(h);
    }
}
template <bool kBF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    return kBF16 ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
}
template <bool kBF16>
__device__ __forceinline__ float load16(const void* p, int64_t i) {
    if constexpr (kBF16)
        return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    else
        return __half2float(static_cast<const __half*>(p)[i]);
}
template <bool kBF16>
__device__ __forceinline__ void store16(void* p, int64_t i, float v) {
    if constexpr (kBF16)
        static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// Values [i, i + 8) of a vector of `n` 16-bit floats at `p` (its element 0
// 16-byte aligned, i a multiple of 8); those at or past n read as 0 and are
// not touched in memory.
template <bool kBF16>
__device__ __forceinline__ void load8_16(const void* p, int64_t i, int64_t n, float (&v)[8]) {
    if (i + 8 <= n) {
        const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = unpack16<kBF16>(x[j]);
            v[2 * j] = f.x;
            v[2 * j + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = i + j < n ? load16<kBF16>(p, i + j) : 0.0f;
    }
}
__device__ __forceinline__ void load8_f32(const float* p, int64_t i, int64_t n, float (&v)[8]) {
    if (i + 8 <= n) {
        const float4 a = *reinterpret_cast<const float4*>(p + i), b = *reinterpret_cast<const float4*>(p + i + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = i + j < n ? p[i + j] : 0.0f;
    }
}
// The same for a vector whose type is known only when the kernel runs.
__device__ __forceinline__ void load8(int kind, const void* p, int64_t i, int64_t n, float (&v)[8]) {
    if (kind == kElemBF16)
        load8_16<true>(p, i, n, v);
    else if (kind == kElemF16)
        load8_16<false>(p, i, n, v);
    else
        load8_f32(static_cast<const float*>(p), i, n, v);
}

// --------------------------------------------------------- the epilogue --

// Lane's row `row`, columns [col, col + 32) of the fp32 sums in r: writes
// them to the saved pre-activations at column `at` (the linear layer's own
// column, or F later for the up half).  Rows of the saved array are 8
// floats' multiples long, so a group of four that starts inside a row's n
// columns stays inside the row.
__device__ __forceinline__ void save_preact(const FfnEpilogue& e, int row, int M, int col, int n, int64_t at,
                                            const uint32_t (&r)[32]) {
    if (row >= M) return;
    float* dst = e.saved + static_cast<int64_t>(row) * e.lds + at;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (col + 4 * j < n) st_global_v4(dst + 4 * j, r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
}

// The linear layer's epilogue on 32 columns of one row: + bias, saved
// pre-activation, activation, + residual (kResid: its ElemKind).
template <int kResid>
__device__ __forceinline__ void linear_epilogue(const FfnEpilogue& e, int row, int M, int col, int n,
                                                uint32_t (&r)[32]) {
    if (e.bias_kind != kElemNone) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float b[8];
            load8(e.bias_kind, e.bias, col + 8 * j, n, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) r[8 * j + i] = __float_as_uint(__uint_as_float(r[8 * j + i]) + b[i]);
        }
    }
    if (e.saved) save_preact(e, row, M, col, n, col, r);
    if (e.act != kActNone) {
        with_act(e.act, [&](auto a) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                r[i] = __float_as_uint(act_value<decltype(a)::value>(__uint_as_float(r[i])));
        });
    }
    if (e.residual && row < M) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float b[8];
            constexpr int64_t kBytes = kResid == kElemF32 ? 4 : 2;
            load8(kResid, static_cast<const char*>(e.residual) + static_cast<int64_t>(row) * e.ldr * kBytes,
                  col + 8 * j, n, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) r[8 * j + i] = __float_as_uint(__uint_as_float(r[8 * j + i]) + b[i]);
        }
    }
}

// The gated layer's on 32 columns: g (gate sums) becomes act(g) * u.
__device__ __forceinline__ void gated_epilogue(const FfnEpilogue& e, int row, int M, int col, int F,
                                               uint32_t (&g)[32], const uint32_t (&u)[32]) {
    if (e.saved) {
        save_preact(e, row, M, col, F, col, g);
        save_preact(e, row, M, col, F, static_cast<int64_t>(F) + col, u);
    }
    with_act(e.act, [&](auto a) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            g[i] = __float_as_uint(act_value<decltype(a)::value>(__uint_as_float(g[i])) * __uint_as_float(u[i]));
    });
}

}  // namespace tsg
