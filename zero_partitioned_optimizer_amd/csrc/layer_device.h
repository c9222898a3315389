// layer_device.h -- device code shared by the layer operators' kernels: the
// counter-based generator of dropout, activations and their derivatives, and
// loads and stores of eight consecutive elements of a row.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layer_internal.h"

namespace zk {

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef v4u v4u_any __attribute__((aligned(2)));        // at any element's address
typedef float v4f __attribute__((ext_vector_type(4)));
typedef v4f v4f_any __attribute__((aligned(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float bf_f(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }
// Two floats to bf16, each rounded once to nearest, ties to even (NaN stays NaN).
__device__ __forceinline__ uint32_t bf_pack(float a, float b) {
    v2bf t;
    t[0] = (__bf16)a;
    t[1] = (__bf16)b;
    return __builtin_bit_cast(uint32_t, t);
}
__device__ __forceinline__ uint16_t bf_one(float a) {
    return __builtin_bit_cast(uint16_t, (__bf16)a);
}

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as
// 1, 2, 3", 2011): ten rounds of two 32 x 32 -> 64 products over a 128-bit counter.
__device__ __forceinline__ v4u philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0,
                                      uint32_t k1) {
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return v4u{c0, c1, c2, c3};
}

// The stream's 64-bit offset: read once per thread, so that a captured call
// draws anew whenever its program has advanced the counter.
__device__ __forceinline__ uint64_t drop_offset(const Drop& d) {
    return d.offset + (d.counter ? (uint64_t)*d.counter : 0);
}

// Dropout of columns 8 * group .. 8 * group + 7 of row `row`: one draw of 128 bits
// gives the eight columns 16 bits each (low half of word k first), which is 1/8 of
// a generator call per element; p is kept to 1 / 65536. Dropped elements become 0
// whatever they held.
__device__ __forceinline__ void drop8(float v[8], const Drop& d, uint64_t off, uint32_t row,
                                      uint32_t group) {
    const v4u w = philox(group, row, (uint32_t)off, (uint32_t)(off >> 32), d.k0, d.k1);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[2 * k] = (w[k] & 0xFFFFu) >= d.thr ? v[2 * k] * d.scale : 0.0f;
        v[2 * k + 1] = (w[k] >> 16) >= d.thr ? v[2 * k + 1] * d.scale : 0.0f;
    }
}

// 1 / (1 + exp(-x)), from the hardware's exp2 and reciprocal (about 1 ulp each).
__device__ __forceinline__ float logistic(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896340736f * x));
}

// tanh-form GELU: z * (1 + tanh(u)) / 2 = z * logistic(2u), u = sqrt(2/pi) (z + 0.044715 z^3).
constexpr float kGelu2C = 1.59576912160573071176f;      // 2 sqrt(2/pi)
constexpr float kGeluA = 0.044715f;

__device__ __forceinline__ float act_of(int32_t act, float z) {
    if (act == ZERO_ACT_RELU) return z < 0.0f ? 0.0f : z;               // NaN stays
    if (act == ZERO_ACT_GELU) return z * logistic(kGelu2C * fmaf(kGeluA * z, z * z, z));
    if (act == ZERO_ACT_SILU) return z * logistic(z);
    return z;
}

// act'(z). Beyond +-128 the logistic is 0 or 1 and the smooth activations' slopes with
// it, and holding z there keeps the formulas' products finite for any z.
__device__ __forceinline__ float act_slope(int32_t act, float z) {
    if (act == ZERO_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;            // 0 at a NaN
    const float h = z > 128.0f ? 128.0f : (z < -128.0f ? -128.0f : z);  // NaN stays
    if (act == ZERO_ACT_GELU) {
        const float s = logistic(kGelu2C * fmaf(kGeluA * h, h * h, h));
        return fmaf(h * s * (1.0f - s), kGelu2C * fmaf(3.0f * kGeluA, h * h, 1.0f), s);
    }
    if (act == ZERO_ACT_SILU) {
        const float s = logistic(h);
        return s * fmaf(h, 1.0f - s, 1.0f);
    }
    return 1.0f;
}

// Up to eight consecutive elements (n of them, the rest 0) from any
// element-aligned address; all eight go as 16-byte accesses.
__device__ __forceinline__ void load8_bf(float v[8], const uint16_t* p, int n) {
    if (n >= 8) {
        const v4u w = *reinterpret_cast<const v4u_any*>(p);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[2 * k] = bf_lo(w[k]);
            v[2 * k + 1] = bf_hi(w[k]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = k < n ? bf_f(p[k]) : 0.0f;
    }
}
__device__ __forceinline__ void load8_f(float v[8], const float* p, int n) {
    if (n >= 8) {
        const v4f a = *reinterpret_cast<const v4f_any*>(p), b = *reinterpret_cast<const v4f_any*>(p + 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] = a[k];
            v[4 + k] = b[k];
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = k < n ? p[k] : 0.0f;
    }
}
__device__ __forceinline__ void store8_bf(uint16_t* p, const float v[8], int n) {
    if (n >= 8) {
        *reinterpret_cast<v4u_any*>(p) =
            v4u{bf_pack(v[0], v[1]), bf_pack(v[2], v[3]), bf_pack(v[4], v[5]), bf_pack(v[6], v[7])};
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) p[k] = bf_one(v[k]);
    }
}
__device__ __forceinline__ void store8_f(float* p, const float v[8], int n) {
    if (n >= 8) {
        *reinterpret_cast<v4f_any*>(p) = v4f{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<v4f_any*>(p + 4) = v4f{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) p[k] = v[k];
    }
}

}  // namespace zk
