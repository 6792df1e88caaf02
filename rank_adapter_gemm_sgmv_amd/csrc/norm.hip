// norm.hip -- what a serving program runs in front of every adapted projection: the residual
// addition and the root-mean-square norm of a batch's rows, written in bf16, in 8 bits with a
// scale per row (the x operand of lora_linear_fp8 or lora_linear_int8), or both, in one pass over
// the data; and rows in 8-bit integers as they are (lora_quant_int8: no norm).
//
//   h = x[m] + residual[m]             (fp32; sum[m] = bf16(h))
//   r = 1 / sqrt(mean(h^2) + eps)      n = h r w
//   y[m] = bf16(n);   s = max(max|n|, 2^-60) / 448;   y8[m] = E4M3(n / s);   y_scale[m] = s
//   8-bit integers: s = max(max|n|, 2^-60) / 127;   y8[m] = rint(127 p / max|p|), p = fp32(h w)
//
// Bound: HBM bytes for many rows, one round trip to memory for few.
//  * A row is read once and stays in registers between its statistics and its output, as
//    fp32 h (never rounded to the bf16 sum first).
//  * Both statistics come from one reduction: r > 0 is the same for the whole row, so
//    max|n| = r max|h w|, and the sum of squares and max|h w| are reduced side by side.  The
//    maximum keeps a NaN (v_maximum3_f32 takes no more instructions than the one that drops it),
//    so that a NaN in weight, or an infinite weight on a zero h, reaches the row's scale.
//  * The 8-bit codes are h w (448 / max|h w|): r cancels, and with it its rounding.
//  * WPR waves share a row, so that a lane holds one to three 16-byte pieces of it and all of
//    the row's loads are in flight at once (one row alone is one round trip to memory).
//  * An integer is the exact rint of a quotient without a division: a product that is right but near a
//    border, and only there the remainder in 64 bits (int8_code).  Memory stays the bound: lora_quant_int8 of
//    4096 x 11008 25.0 us (135 MB: 5.4 TB/s, a large copy's rate on the same card 5.2-5.6), lora_rmsnorm_int8 of
//    1 x 4096 3.2 us on the GPU, 6.0 per call.
#include "common.h"

namespace lora {

namespace {

// What the rows' 8-bit output is: E4M3 codes, integers, or integers of x itself (no norm).
enum Rows8 { kE4m3, kInt8, kInt8Plain };

template <Rows8 Q>
constexpr float kTop8 = Q == kE4m3 ? 448.0f : 127.0f;  // the largest value of an 8-bit code
constexpr float kFloor8 = 0x1p-60f;                  // rows of zeros still get a normal scale
constexpr float kShrink = 0x1p-80f;                  // rescales rows whose squares overflow

// h w (448 / max|h w|) -> four codes of one dword
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}

// rint(127 p / top), ties to even, exactly.  q0 = p (127 / top) is off by at most 2^-23 of itself, so by 2^-16,
// and only quotients within 2^-11 of a border take the exact remainder: one in a thousand, three to five in a
// thousand of bf16 rows as they are, whose short significands make ties.  p is not above top; a NaN gives 0.
__device__ __forceinline__ int int8_code(float p, float f, float top) {
    const float q0 = p * f;
    float k = rintf(q0);
    if (fabsf(q0 - k) > 0.4995f) {
        const double e = 127.0 * (double)p - (double)k * (double)top, half = 0.5 * (double)top;
        const bool odd = ((int)k & 1) != 0;
        if (e > half || (e == half && odd)) k += 1.0f;
        if (e < -half || (e == -half && odd)) k -= 1.0f;
    }
    return k == k ? (int)k : 0;
}
__device__ __forceinline__ uint32_t pack_int8x4(int a, int b, int c, int d) {
    return (uint32_t)(a & 255) | (uint32_t)(b & 255) << 8 | (uint32_t)(c & 255) << 16 | (uint32_t)d << 24;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
    return v;
}
// the larger of a and b, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v = max_nan(v, __shfl_xor(v, d, 64));
    return v;
}

// h of one 16-byte piece: x, plus the residual when there is one
__device__ __forceinline__ void norm_h8(float h[8], uint4 x, uint4 res, bool has_res) {
    unpack8(x, h);
    if (has_res) {
        float q[8];
        unpack8(res, q);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] += q[e];
    }
}

// Row statistics -> factors of the outputs: y = (h r) w, code = ((h q) w) f, scale s.  Integers are
// rint(127 (h q) w / top).
struct NormFactors {
    float r, q, f, s, top;
};
// top: max|h w|, or (nw: that overflowed) max|n| itself
template <Rows8 Q>
__device__ __forceinline__ NormFactors norm_factors(float r, float top, bool nw) {
    NormFactors o;
    const float q = nw ? 1.0f : r, mx = q * top;
    o.r = r;
    o.q = nw ? r : 1.0f;
    o.s = fmaxf(mx, kFloor8) / kTop8<Q>;
    // (below the floor the codes are n / s with the floor's s; above it r cancels)
    o.f = mx > kFloor8 ? kTop8<Q> / top : q / o.s;
    o.top = mx > kFloor8 ? top : kFloor8 / q;
    // a row with an infinity (r = 0) or a NaN, in h or in h w, has no scale: all its codes are NaN
    // (integers 0)
    if (!(mx < __builtin_inff()) || !(r > 0.0f)) o.s = o.f = __builtin_nanf("");
    return o;
}

// Outputs are written past the caches' reuse order (nontemporal): a row is not read again here,
// and the reader that follows takes it from memory's own cache.  Residual, sum and both
// outputs at d 4096, plain stores -> these: 10.7 -> 8.3 us at 1024 rows, 54.0 -> 51.8 us at
// 8192 (5.8 TB/s; a large copy reaches 5.5), the same at 64 rows and below.
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void st_bf16x8(uint16_t *p, const float f[8]) {
    st16_nt(p, make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]),
                          cvt_bf16x2(f[6], f[7])));
}

template <Rows8 Q>
__device__ __forceinline__ void norm_store8(const NormArgs &a, size_t at, const float h[8],
                                            uint4 w, const NormFactors &nf) {
    if (a.sum) st_bf16x8(a.sum + at, h);
    float g[8], n[8];
    unpack8(w, g);
    if (a.y) {
        // |h r| is at most sqrt(d), so that no product overflows where n does not
#pragma unroll
        for (int e = 0; e < 8; ++e) n[e] = h[e] * nf.r * g[e];
        st_bf16x8(a.y + at, n);
    }
    if (a.y8) {
        u32x2_t v;
        if constexpr (Q == kE4m3) {
#pragma unroll
            for (int e = 0; e < 8; ++e) n[e] = h[e] * nf.q * g[e] * nf.f;
            v = {pack_e4m3x4(n[0], n[1], n[2], n[3]), pack_e4m3x4(n[4], n[5], n[6], n[7])};
        } else {
            int c[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) c[e] = int8_code(h[e] * nf.q * g[e], nf.f, nf.top);
            v = {pack_int8x4(c[0], c[1], c[2], c[3]), pack_int8x4(c[4], c[5], c[6], c[7])};
        }
        __builtin_nontemporal_store(v, reinterpret_cast<u32x2_t *>(a.y8 + at));
    }
}

constexpr uint32_t kOneBf16x2 = 0x3F803F80u;  // (1, 1): the weight when none is given

// Waves of one row add their (sum of squares, max|h w|) in wave order.  Every thread of the
// block must call it.
template <int WPR>
__device__ __forceinline__ void row_reduce(float &ss, float &top, float (*red)[2], int wave) {
    ss = wave_sum(ss);
    top = wave_max(top);
    if constexpr (WPR > 1) {
        if ((threadIdx.x & 63) == 0) { red[wave][0] = ss; red[wave][1] = top; }
        __syncthreads();
        const int w0 = wave / WPR * WPR;
        ss = red[w0][0];
        top = red[w0][1];
#pragma unroll
        for (int i = 1; i < WPR; ++i) {
            ss += red[w0 + i][0];
            top = max_nan(top, red[w0 + i][1]);
        }
    }
}

// WPR waves per row, VPL 16-byte pieces per lane: rows of at most 512 WPR VPL elements.
template <Rows8 Q, int WPR, int VPL>
__global__ __launch_bounds__(WPR > 4 ? WPR * 64 : 256) void rmsnorm_kernel(NormArgs a) {
    constexpr int NW = WPR > 4 ? WPR : 4;  // waves per block
    constexpr int RPB = NW / WPR;          // rows per block
    __shared__ float red[NW][2], red2[NW][2], red3[NW][2];
    const int wave = threadIdx.x >> 6;
    const int row = blockIdx.x * RPB + wave / WPR;
    const bool live = row < a.M;
    const int m = live ? row : a.M - 1;  // (spare waves repeat the last row and store nothing)
    const int c0 = ((wave % WPR) * 64 + (threadIdx.x & 63)) * 8;
    const size_t base = (size_t)m * a.d;
    const bool has_res = a.residual != nullptr;

    uint4 xv[VPL], rv[VPL], wv[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int c = min(c0 + i * (WPR * 512), a.d - 8);
        xv[i] = ld16(a.x + base + c);
        rv[i] = has_res ? ld16(a.residual + base + c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        wv[i] = a.weight ? ld16(a.weight + min(c0 + i * (WPR * 512), a.d - 8))
                         : make_uint4(kOneBf16x2, kOneBf16x2, kOneBf16x2, kOneBf16x2);

    float h[VPL][8], ss = 0.0f, top = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        norm_h8(h[i], xv[i], rv[i], has_res);
        if (c0 + i * (WPR * 512) < a.d) {
            float g[8];
            unpack8(wv[i], g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ss = fmaf(h[i][e], h[i][e], ss);
                top = max_nan(top, fabsf(h[i][e] * g[e]));
            }
        }
    }
    row_reduce<WPR>(ss, top, red, wave);
    const float ms = Q == kInt8Plain ? 1.0f : ss / (float)a.d + a.eps;
    float r = 1.0f / sqrtf(ms);
    // Rows at the ends of the range go on: their branches are uniform in the row, so in the wave
    // (WPR == 1) or the block (its barriers).
    static_assert(WPR == 1 || RPB == 1, "a block with barriers holds one row");
    if (!(ms < __builtin_inff())) {  // some square overflowed: once more on h 2^-80
        float s2 = 0.0f, t2 = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (c0 + i * (WPR * 512) < a.d)
#pragma unroll
                for (int e = 0; e < 8; ++e) s2 = fmaf(h[i][e] * kShrink, h[i][e] * kShrink, s2);
        row_reduce<WPR>(s2, t2, red2, wave);
        r = kShrink / sqrtf(s2 / (float)a.d + a.eps * kShrink * kShrink);
    }
    const bool nw = Q != kInt8Plain && !(top < __builtin_inff());
    if (nw) {  // some h w did: max|n| instead
        float s3 = 0.0f;
        top = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (c0 + i * (WPR * 512) < a.d) {
                float g[8];
                unpack8(wv[i], g);
#pragma unroll
                for (int e = 0; e < 8; ++e) top = max_nan(top, fabsf(h[i][e] * r * g[e]));
            }
        row_reduce<WPR>(s3, top, red3, wave);
    }
    if (!live) return;
    const NormFactors nf = norm_factors<Q>(r, top, nw);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int c = c0 + i * (WPR * 512);
        if (c < a.d) norm_store8<Q>(a, base + c, h[i], wv[i], nf);
    }
    if (a.y_scale && c0 == 0) a.y_scale[m] = nf.s;
}

// Rows too long for registers: one block of 16 waves per row, which it reads twice (the second
// time mostly from L2).
template <Rows8 Q>
__global__ __launch_bounds__(1024) void rmsnorm_long_kernel(NormArgs a) {
    __shared__ float red[16][2], red2[16][2], red3[16][2];
    const int wave = threadIdx.x >> 6;
    const size_t base = (size_t)blockIdx.x * a.d;
    const bool has_res = a.residual != nullptr;
    const uint4 one = make_uint4(kOneBf16x2, kOneBf16x2, kOneBf16x2, kOneBf16x2);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    // the row's sum of (h k)^2 and max|h q w|
    auto stats = [&](float k, float q, float &ss, float &top) {
        ss = top = 0.0f;
        for (int c = threadIdx.x * 8; c < a.d; c += 8192) {
            float h[8], g[8];
            norm_h8(h, ld16(a.x + base + c), has_res ? ld16(a.residual + base + c) : zero, has_res);
            unpack8(a.weight ? ld16(a.weight + c) : one, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ss = fmaf(h[e] * k, h[e] * k, ss);
                top = max_nan(top, fabsf(h[e] * q * g[e]));
            }
        }
    };
    float ss, top, spare;
    stats(1.0f, 1.0f, ss, top);
    row_reduce<16>(ss, top, red, wave);
    const float ms = Q == kInt8Plain ? 1.0f : ss / (float)a.d + a.eps;
    float r = 1.0f / sqrtf(ms);
    if (!(ms < __builtin_inff())) {  // uniform in the block, as the next one
        stats(kShrink, 1.0f, ss, spare);
        row_reduce<16>(ss, spare, red2, wave);
        r = kShrink / sqrtf(ss / (float)a.d + a.eps * kShrink * kShrink);
    }
    const bool nw = Q != kInt8Plain && !(top < __builtin_inff());
    if (nw) {
        stats(1.0f, r, spare, top);
        row_reduce<16>(spare, top, red3, wave);
    }
    const NormFactors nf = norm_factors<Q>(r, top, nw);
    for (int c = threadIdx.x * 8; c < a.d; c += 8192) {
        float h[8];
        norm_h8(h, ld16(a.x + base + c), has_res ? ld16(a.residual + base + c) : zero, has_res);
        norm_store8<Q>(a, base + c, h, a.weight ? ld16(a.weight + c) : one, nf);
    }
    if (a.y_scale && threadIdx.x == 0) a.y_scale[blockIdx.x] = nf.s;
}

template <Rows8 Q, int WPR, int VPL>
void launch_one(const NormArgs &a, hipStream_t s) {
    constexpr int NW = WPR > 4 ? WPR : 4;
    constexpr int RPB = NW / WPR;
    launch((rmsnorm_kernel<Q, WPR, VPL>), dim3((unsigned)((a.M + RPB - 1) / RPB)), dim3(64 * NW), 0, s, a);
}

}  // namespace

// Waves per row x pieces per lane, all outputs, us per launch inside a graph:
//   d 1024  4 x 1: 2.64 at 1 row, 3.12 at 256, 5.22 at 1024, 11.98 at 4096
//           1 x 2: 2.95           3.35         5.00          10.50
//   d 4096  8 x 1: 2.95 at 1 row, 4.88 at 256, 30.3 at 4096, 103.7 at 16384 (5.8 TB/s)
//           4 x 2: 3.14           5.13         31.6          106.0
//           1 x 8: 6.04           7.88         37.2          120.1
//           16 x 1: 3.28          5.20         34.1          126.3
//   d 8192  8 x 2: 3.72 at 1 row, 56.8 at 4096;  16 x 1: 3.81, 58.1;  4 x 4: 4.12, 59.8
//   d 11008 8 x 3: 4.43 at 1 row, 75.9 at 4096;  16 x 2: 4.58, 92.1
// so eight waves share a row wherever it has a piece for each of their lanes, and only rows of
// 513-1024 elements go by the number of rows.
template <Rows8 Q>
static void launch_rows(const NormArgs &a, hipStream_t s) {
    if (a.d <= 512) launch_one<Q, 1, 1>(a, s);
    else if (a.d <= 1024 && a.M >= 1024) launch_one<Q, 1, 2>(a, s);
    else if (a.d <= 2048) launch_one<Q, 4, 1>(a, s);
    else if (a.d <= 4096) launch_one<Q, 8, 1>(a, s);
    else if (a.d <= 8192) launch_one<Q, 8, 2>(a, s);
    else if (a.d <= 12288) launch_one<Q, 8, 3>(a, s);
    else if (a.d <= 16384) launch_one<Q, 16, 2>(a, s);
    else launch(rmsnorm_long_kernel<Q>, dim3((unsigned)a.M), dim3(1024), 0, s, a);
}

// A launch holds fewer than 2^32 threads: LORA_MAX_ROWS = 2^22 rows on blocks of 1024 are one too
// many, so rows go in parts of 2^21 (rows are independent).
hipError_t launch_rmsnorm(const NormArgs &a, hipStream_t s) {
    constexpr int kPart = 1 << 21;
    for (int m = 0; m < a.M; m += kPart) {
        NormArgs p = a;
        const size_t at = (size_t)m * a.d;
        p.M = a.M - m < kPart ? a.M - m : kPart;
        p.x = a.x + at;
        if (a.residual) p.residual = a.residual + at;
        if (a.sum) p.sum = a.sum + at;
        if (a.y) p.y = a.y + at;
        if (a.y8) {
            p.y8 = a.y8 + at;
            p.y_scale = a.y_scale + m;
        }
        if (!a.int8) launch_rows<kE4m3>(p, s);
        else if (a.norm) launch_rows<kInt8>(p, s);
        else launch_rows<kInt8Plain>(p, s);
    }
    return hipGetLastError();
}

}  // namespace lora
