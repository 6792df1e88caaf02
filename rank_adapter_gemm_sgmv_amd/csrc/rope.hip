// rope.hip -- rotary positions of a batch's queries and keys (lora_rope): what stands between the
// q and k projections and attention.
//
//   (a, b) -> factor (a cos t - b sin t, a sin t + b cos t),   t = 2 pi frac(positions[m] freqs[i])
//
// for pair i of each head's first rot_dim elements: (i, i + rot_dim / 2), or (2 i, 2 i + 1)
// interleaved; inverse turns by -t.  Elements past rot_dim pass through.
//
// Bound: HBM bytes for many rows (each element read and written once), one round trip for few.
//  * positions[m] freqs[i] and its fraction are 64-bit: a position of a million has angles of 10^5
//    turns, of which fp32 would keep two or three digits of the fraction.  What is left (an eighth of a
//    turn either way) goes to fp32 polynomials.
//  * A block turns its rows' rot_dim / 2 angles into cosines and sines once, in LDS, and all heads of
//    the row share them; every thread then takes 16-byte pieces of a head, both halves of its
//    pairs, so that an in-place call reads what it writes before anyone writes it.
//  * A row per block, so that many rows' tables and loads overlap; few rows of many heads are cut over
//    several blocks, each with a table of its own (4 rows of 128 heads of 256: 41.3 us in a block per
//    row, 4.6 in several).  Four items ahead in registers took 80.6 us at 8192 rows, where one at a time takes
//    33.1 (40 heads of 128 in bf16, 168 MB: 5.1 TB/s); one row 2.4 us on the GPU, 7.3 per call.
#include <type_traits>

#include "common.h"

namespace lora {

namespace {

constexpr int kThreadsRope = 256;
constexpr int kTableMax = LORA_ROPE_MAX_DIM / 2;  // (cos, sin) pairs of a row

// cos and sin of 2 pi t, both times factor.  |t - its quarter| <= 1/8, where the Taylor polynomials
// of degree 9 and 10 are within 2e-9 of the functions.
__device__ __forceinline__ float2 turn_cos_sin(double t, float factor, float way) {
    t -= rint(t);
    const double quarter = rint(4.0 * t);
    const float x = (float)(t - 0.25 * quarter) * 6.28318530717958648f, x2 = x * x;
    const float s = x * fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), 1.0f);
    const float c = fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
    const int k = (int)quarter & 3;
    const float cc = k == 0 ? c : k == 1 ? -s : k == 2 ? -c : s;
    const float ss = k == 0 ? s : k == 1 ? c : k == 2 ? -s : -c;
    return make_float2(cc * factor, ss * factor * way);
}

// One 16-byte piece as fp32 values (eight bf16, or four fp32), and back.
template <bool F32>
struct Piece {
    static constexpr int N = F32 ? 4 : 8;
    float v[N];
    __device__ __forceinline__ void load(const uint4 u) {
        if constexpr (F32) {
            v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y);
            v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
        } else {
            unpack8(u, v);
        }
    }
    __device__ __forceinline__ uint4 store() const {
        if constexpr (F32)
            return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        else
            return make_uint4(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]), cvt_bf16x2(v[4], v[5]), cvt_bf16x2(v[6], v[7]));
    }
};

template <bool F32>
__device__ __forceinline__ float ld_el(const char *p) {
    if constexpr (F32) return *reinterpret_cast<const float *>(p);
    else return bf16_lo(*reinterpret_cast<const uint16_t *>(p));
}
template <bool F32>
__device__ __forceinline__ void st_el(char *p, float v) {
    if constexpr (F32) *reinterpret_cast<float *>(p) = v;
    else *reinterpret_cast<uint16_t *>(p) = (uint16_t)f32_to_bf16_rne(v);
}

// n / d for n d < 2^32: a product with 2^32 / d rounded up (0 stands for d = 1).
struct Divisor {
    uint32_t d, inv;
    explicit Divisor(uint32_t n) : d(n), inv(n > 1 ? 0xFFFFFFFFu / n + 1u : 0u) {}
    __device__ __forceinline__ int of(int n) const { return inv ? (int)__umulhi((uint32_t)n, inv) : n; }
};

// Block (row, heads h0 .. h0 + heads of q's and k's laid end to end).  A head is n_all items: its pairs,
// then what passes through.  VEC: pairs go in whole 16-byte pieces; else pair by pair.
template <bool F32, bool VEC, bool INTER>
__global__ __launch_bounds__(kThreadsRope) void rope_kernel(RopeArgs a, int heads, int n_rot, Divisor n_all) {
    constexpr int EL = F32 ? 4 : 2, V = 16 / EL;
    __shared__ float2 tab[kTableMax];
    const int tid = threadIdx.x, half = a.rot_dim / 2;
    const int64_t row = blockIdx.x;
    const int h0 = blockIdx.y * heads, nh = min(heads, a.q.heads + a.k.heads - h0);
    const double pos = a.positions[row];
    for (int i = tid; i < half; i += kThreadsRope)
        tab[i] = turn_cos_sin(pos * a.freqs[i], a.factor, a.inverse ? -1.0f : 1.0f);
    __syncthreads();
    const float2 *const cs = tab;
    const int items = nh * (int)n_all.d;
    for (int it = tid; it < items; it += kThreadsRope) {
        const int head = n_all.of(it), i = it - head * (int)n_all.d, h = h0 + head;
        const bool is_q = h < a.q.heads;
        const RopeHeads &t = is_q ? a.q : a.k;
        const int hh = is_q ? h : h - a.q.heads;
        const char *x = static_cast<const char *>(t.x) + (row * t.x_stride + (int64_t)hh * a.head_dim) * EL;
        char *y = static_cast<char *>(t.y) + (row * t.y_stride + (int64_t)hh * a.head_dim) * EL;
        if constexpr (VEC) {
            if (i >= n_rot) {
                const int at = (a.rot_dim + (i - n_rot) * V) * EL;
                if (x != y) st16(y + at, ld16(x + at));
            } else if constexpr (INTER) {
                Piece<F32> p, o;
                p.load(ld16(x + i * 16));
#pragma unroll
                for (int e = 0; e < V / 2; ++e) {
                    const float2 w = cs[i * (V / 2) + e];
                    o.v[2 * e] = p.v[2 * e] * w.x - p.v[2 * e + 1] * w.y;
                    o.v[2 * e + 1] = p.v[2 * e] * w.y + p.v[2 * e + 1] * w.x;
                }
                st16(y + i * 16, o.store());
            } else {
                Piece<F32> p, q, o, u;
                p.load(ld16(x + i * 16));
                q.load(ld16(x + half * EL + i * 16));
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float2 w = cs[i * V + e];
                    o.v[e] = p.v[e] * w.x - q.v[e] * w.y;
                    u.v[e] = p.v[e] * w.y + q.v[e] * w.x;
                }
                st16(y + i * 16, o.store());
                st16(y + half * EL + i * 16, u.store());
            }
        } else {
            if (i >= n_rot) {
                // (as bits: a conversion would quiet a NaN)
                using Two = std::conditional_t<F32, uint2, uint32_t>;
                const int at = (a.rot_dim + (i - n_rot) * 2) * EL;
                if (x != y) *reinterpret_cast<Two *>(y + at) = *reinterpret_cast<const Two *>(x + at);
                continue;
            }
            const int pa = (INTER ? 2 * i : i) * EL, pb = (INTER ? 2 * i + 1 : i + half) * EL;
            const float va = ld_el<F32>(x + pa), vb = ld_el<F32>(x + pb);
            const float2 w = cs[i];
            st_el<F32>(y + pa, va * w.x - vb * w.y);
            st_el<F32>(y + pb, va * w.y + vb * w.x);
        }
    }
}

}  // namespace

hipError_t launch_rope(const RopeArgs &a, hipStream_t s) {
    const int V = a.f32 ? 4 : 8, half = a.rot_dim / 2, n_heads = a.q.heads + a.k.heads;
    if (a.M < 1 || n_heads < 1 || half < 1 || half > kTableMax || a.head_dim % 8 != 0) return hipErrorInvalidValue;
    const bool vec = (a.interleaved ? a.rot_dim % V : half % V) == 0;
    const int n_rot = vec ? (a.interleaved ? a.rot_dim / V : half / V) : half;
    const int n_all = n_rot + (a.head_dim - a.rot_dim) / (vec ? V : 2);
    // a block per row; few rows of many items take more blocks, four items a thread
    int heads = n_heads;
    if (a.M < 512 && n_heads * n_all > 4 * kThreadsRope) heads = n_all < 4 * kThreadsRope ? 4 * kThreadsRope / n_all : 1;
    const dim3 grid((unsigned)a.M, (unsigned)((n_heads + heads - 1) / heads));
#define ROPE_ONE(F, VE, IN) launch((rope_kernel<F, VE, IN>), grid, dim3(kThreadsRope), 0, s, a, heads, n_rot, Divisor((uint32_t)n_all))
#define ROPE_VEC(F, VE)                                                                        \
    if (a.interleaved) ROPE_ONE(F, VE, true);                                                  \
    else ROPE_ONE(F, VE, false)
#define ROPE_TYPE(F)                                                                           \
    if (vec) {                                                                                 \
        ROPE_VEC(F, true);                                                                     \
    } else {                                                                                   \
        ROPE_VEC(F, false);                                                                    \
    }
    if (a.f32) {
        ROPE_TYPE(true)
    } else {
        ROPE_TYPE(false)
    }
#undef ROPE_TYPE
#undef ROPE_VEC
#undef ROPE_ONE
    return hipGetLastError();
}

}  // namespace lora
