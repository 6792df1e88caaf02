// epilogue.h -- what follows a projection in the same pass that rounds y (lora_linear_act,
// lora_linear_fp8):
//
//   y = act(row_scale[m] z + bias) * mul + residual        (fp32, one rounding)
//
// z is x W plus the adapter's delta.  Every kernel that writes y applies it where the fp32 sum
// is still in registers, so the four optional operands cost their own bytes and nothing else.
//
// Activations use the hardware's exp2 and reciprocal (about 1 ulp each); exp's argument is
// rounded once, a relative error of |z| 2^-24 in e^z where e^z matters (|z| of a few).  GELU's
// Gaussian is Abramowitz and Stegun 7.1.26 in its erfc form, |error| <= 1.5e-7: the library's
// erf costs three times the instructions, which a prefill tile cannot hide behind MFMAs (its
// epilogue runs after the last of them).
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

__device__ __forceinline__ float epi_sigmoid(float z) {  // 1 / (1 + e^-z); 0 where e^-z overflows
    return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

// Phi(z), the standard normal distribution: erfc(|u|) / 2 on one side, its complement on the
// other, u = z / sqrt(2)
__device__ __forceinline__ float epi_normal_cdf(float z) {
    const float u = fabsf(z) * 0.70710678118654752f;
    const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f, u, 1.0f));
    float p = fmaf(1.061405429f, t, -1.453152027f);
    p = fmaf(p, t, 1.421413741f);
    p = fmaf(p, t, -0.284496736f);
    p = fmaf(p, t, 0.254829592f);
    const float half = 0.5f * p * t * __expf(-u * u);
    return z < 0.0f ? half : 1.0f - half;
}

// SiLU is z sigmoid(z), the tanh form of GELU z sigmoid(2 sqrt(2 / pi) (z + 0.044715 z^3)),
// since (1 + tanh v) / 2 = sigmoid(2 v): one code for both, with c the cubic's coefficients.
__device__ __forceinline__ float epi_act(float z, int act) {
    if (act == LORA_ACT_RELU) return z < 0.0f ? 0.0f : z;  // (a NaN stays one)
    if (act == LORA_ACT_GELU) return z * epi_normal_cdf(z);
    const float c1 = act == LORA_ACT_SILU ? 1.0f : 1.5957691216057308f;
    const float c3 = act == LORA_ACT_SILU ? 0.0f : 0.071354816272600f;
    return z * epi_sigmoid(fmaf(c3 * z * z, z, c1 * z));
}

// The operands of V consecutive elements of one row, loaded ahead of their use.
template <int V, bool YF32>
struct EpiOperands {
    static constexpr int YW = YF32 ? V : V / 2;
    uint32_t b[V / 2], mu[YW], re[YW];
    float rs;

    __device__ __forceinline__ void load(const Epilogue &e, int m, int n, int N) {
        const size_t at = ((size_t)m * N + n) * (YF32 ? 4 : 2);
        rs = e.row_scale ? e.row_scale[m] : 1.0f;
        if (e.bias) ld_words(b, e.bias + n);
        if (e.mul) ld_words(mu, static_cast<const char *>(e.mul) + at);
        if (e.residual) ld_words(re, static_cast<const char *>(e.residual) + at);
    }
    static __device__ __forceinline__ float of(const uint32_t (&w)[YW], int i) {
        if constexpr (YF32) return __uint_as_float(w[i]);
        else return (i & 1) ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
    }
    // z -> y, element by element
    __device__ __forceinline__ void apply(const Epilogue &e, float (&z)[V]) const {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (e.row_scale) z[i] *= rs;
            if (e.bias) z[i] += (i & 1) ? bf16_hi(b[i / 2]) : bf16_lo(b[i / 2]);
        }
        if (e.act != LORA_ACT_NONE) {
#pragma unroll
            for (int i = 0; i < V; ++i) z[i] = epi_act(z[i], e.act);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (e.mul) z[i] *= of(mu, i);
            if (e.residual) z[i] += of(re, i);
        }
    }
};

}  // namespace lora
