// epilogue.h -- what follows a projection in the same pass that rounds y (lora_linear_act,
// lora_linear_fp8):
//
//   y = act(row_scale[m] z + bias) * mul + residual        (fp32, one rounding)
//
// z is x W plus the adapter's delta.  Every kernel that writes y applies it where the fp32 sum
// is still in registers, so the four optional operands cost their own bytes and nothing else.
//
// Activations use the hardware's exp2 and reciprocal (about 1 ulp each); exp2's argument is
// rounded once or twice, a relative error of |z| 2^-23 in e^z.
// GELU's Gaussian tail is a polynomial fitted here (epi_gelu): the library's erf costs three times
// the instructions, which a prefill tile cannot hide behind MFMAs (its epilogue runs after the last of
// them).
#pragma once

#include "common.h"

namespace lora {

// W consecutive dwords (W a power of two), p aligned to min(4 W, 16) bytes
template <int W>
__device__ __forceinline__ void ld_words(uint32_t (&r)[W], const void *p) {
    if constexpr (W >= 4) {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
            r[4 * i] = v.x; r[4 * i + 1] = v.y; r[4 * i + 2] = v.z; r[4 * i + 3] = v.w;
        }
    } else if constexpr (W == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        r[0] = v.x; r[1] = v.y;
    } else {
        r[0] = *reinterpret_cast<const uint32_t *>(p);
    }
}

constexpr float kLog2e = 1.4426950408889634f;

// z / (1 + e^-z); e^-z overflows to a factor of 0
__device__ __forceinline__ float epi_silu(float z) {
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * z));
}

// z (1 + tanh v) / 2 = z / (1 + e^-2v), v = sqrt(2 / pi) (z + 0.044715 z^3)
__device__ __forceinline__ float epi_gelu_tanh(float z) {
    constexpr float c1 = -2.0f * 0.79788456080286536f * kLog2e;
    const float e = __builtin_amdgcn_exp2f(z * fmaf(0.044715f * c1, z * z, c1));
    return z * __builtin_amdgcn_rcpf(1.0f + e);
}

// z Phi(z) = max(z, 0) - |z| Phi(-|z|), with Phi(-a) = t P(t) e^(-a^2 / 2), t = 1 / (1 + 0.275 a).
// P is the polynomial of degree 8 whose t P(t) has the smallest largest relative error against
// erfcx(a / sqrt(2)) / 2 over 0 <= a <= 40 (4.3e-8; a linear programme over its values), so that
// the tail of a negative z is right to its own size: the result is within (24 + 1.5 z^2) 2^-24 of it
// (t 3 units, up to 2.9 times in P; P 4; products and exp2 6; exp2's argument 1.25 z^2).  One term less
// is off by 6.4e-7, one of five terms with an absolute bound (1.5e-7) was off by 5e-5 at z = -3 and 4e-3
// at -6.  +infinity keeps a finite factor against e^-inf = 0; -infinity gives NaN, as z Phi(z) does.
__device__ __forceinline__ float epi_gelu(float z) {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.275f, fabsf(z), 1.0f));
    float p = fmaf(0.027061667f, t, -0.110292655f);
    p = fmaf(p, t, 0.129608795f);
    p = fmaf(p, t, -0.0347237383f);
    p = fmaf(p, t, 0.0878079468f);
    p = fmaf(p, t, 0.0789904468f);
    p = fmaf(p, t, 0.102181808f);
    p = fmaf(p, t, 0.109655047f);
    p = fmaf(p, t, 0.109710667f);
    const float tail = p * t * __builtin_amdgcn_exp2f(-0.5f * kLog2e * z * z);
    return fmaf(-fabsf(fminf(z, 3e38f)), tail, fmaxf(z, 0.0f));
}

// The activation of V elements (one branch for all of them).
template <int V>
__device__ __forceinline__ void epi_act(float (&z)[V], int act) {
    if (act == LORA_ACT_NONE) return;
    if (act == LORA_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = epi_silu(z[i]);
    } else if (act == LORA_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = epi_gelu(z[i]);
    } else if (act == LORA_ACT_GELU_TANH) {
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = epi_gelu_tanh(z[i]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = z[i] < 0.0f ? 0.0f : z[i];  // (a NaN stays one)
    }
}

// The operands of V consecutive elements of one row, loaded ahead of their use.
template <int V, bool YF32>
struct EpiOperands {
    static constexpr int YW = YF32 ? V : V / 2;
    uint32_t b[V / 2], mu[YW], re[YW];
    float rs;

    __device__ __forceinline__ void load(const Epilogue &e, int m, int n, int N) {
        rs = e.row_scale ? e.row_scale[m] : 1.0f;
        load_bias(e, n);
        load_row(e, m, n, N);
    }
    __device__ __forceinline__ void load_bias(const Epilogue &e, int n) {
        if (e.bias) ld_words(b, e.bias + n);
    }
    __device__ __forceinline__ void load_row(const Epilogue &e, int m, int n, int N) {
        const size_t at = ((size_t)m * N + n) * (YF32 ? 4 : 2);
        if (e.mul) ld_words(mu, static_cast<const char *>(e.mul) + at);
        if (e.residual) ld_words(re, static_cast<const char *>(e.residual) + at);
    }
    static __device__ __forceinline__ float of(const uint32_t (&w)[YW], int i) {
        if constexpr (YF32) return __uint_as_float(w[i]);
        else return (i & 1) ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
    }
    // z -> y, element by element
    __device__ __forceinline__ void apply(const Epilogue &e, float (&z)[V]) const {
        if (e.row_scale) {
#pragma unroll
            for (int i = 0; i < V; ++i) z[i] *= rs;
        }
        if (e.bias) {
#pragma unroll
            for (int i = 0; i < V; ++i) z[i] += (i & 1) ? bf16_hi(b[i / 2]) : bf16_lo(b[i / 2]);
        }
        epi_act<V>(z, e.act);
        if (e.mul) {
#pragma unroll
            for (int i = 0; i < V; ++i) z[i] *= of(mu, i);
        }
        if (e.residual) {
#pragma unroll
            for (int i = 0; i < V; ++i) z[i] += of(re, i);
        }
    }
};

}  // namespace lora
