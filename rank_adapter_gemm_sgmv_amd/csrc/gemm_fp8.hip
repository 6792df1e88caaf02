// gemm_fp8.hip -- z = (x8 W8^T) w_scale on 8-bit operands: E4M3 codes with fp32 sums, for
// lora_linear_fp8, or integers with int32 sums, for lora_linear_int8: x8[M][K] with a scale per row
// (applied with the epilogue), W8[N][K] with a scale per column.
//
// gfx950 design
//  * v_mfma_f32_32x32x64_f8f6f4: 64 k per instruction at twice the bf16 rate (its unscaled form:
//    the scales here belong to rows and columns, not to blocks of 32 k).
//  * The tiles and waves of the bf16 kernel (gemm_big.hip).  A stage is 128 k of both operands: a
//    row of it is one whole 128-byte line, and a direct global->LDS load covers eight rows.  A
//    load costs the CU by the lines it touches: with stages of 64 k (four in a ring, every load
//    16 half lines) the same K loop took 201 us at 4096 x 4096 x 11008, now 145 us (2.55 PFLOP/s;
//    MFMAs alone reach 3.9 on random codes, which the card's power allows).  Two stages in LDS,
//    one multiplied while the other is loaded.
//  * W8 lies as x8 does (K contiguous), so both are staged alike, 16-byte chunk c of row r at
//    c ^ ((r / 2) % 8), and read with ds_read_b128: 16 rows of one chunk meet all 64 banks once.
//  * That instruction's adder aligns the eight products of an octet of k to the largest of them and
//    drops what lies 14 or more binary places below (measured: of 2^12 + 2^(12 - d) - 2^12 the
//    second term survives to d = 13; between octets, and into the sum, to d = 23).  On random
//    codes the result is off by 1.6e-5 of its size (4096 k), a hundredth of y's own rounding to
//    bf16; the quantisation of x8 moved it by 4e-2.  A caller who asks for y in fp32 gets sums
//    whose products are all kept: the codes widened to bf16 (exact) on v_mfma_f32_32x32x16_bf16,
//    at half the rate (the 8-bit 32x32x16 instruction has the same adder).
//  * A lane's 32 codes of an operand are chunks g and g + 2 of its row (g = lane / 32).  Which k
//    they are does not matter as long as both operands agree, as the MFMA pairs equal places.
//  * Integers: v_mfma_i32_32x32x32_i8 takes a lane's 16-byte chunk as it lies, half the k of the E4M3
//    instruction at the same rate per k, and sums exactly, so y in fp32 needs no second form.  4096 x 11008 x
//    4096 172 us in the GEMM (2.15 POP/s with delta, epilogue and store; a library product of 4096^3 2.07, of
//    8192^3 2.52).
//  * Enough tiles to fill the chip: rows in segment order, the LoRA delta as extra bf16 MFMA
//    steps, then the epilogue and the only store (big_tiles.h).  Fewer: K is split over ks
//    workgroups per tile, which write scaled fp32 slices [ks][M][N]; the reduction that follows
//    (launch_splitk_reduce_lora) adds them, the delta and the epilogue.
#include <type_traits>

#include "big_tiles.h"

namespace lora {

namespace {

constexpr int kK8 = 128;  // k per stage: two MFMA steps

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

// The K loop's sums: fp32, or exact int32 for integers.
template <bool INT>
using Sum8 = std::conditional_t<INT, i32x16_t, f32x16_t>;

template <class C>
struct Frags8 {
    i32x8_t a[C::TM];
    i32x8_t b[C::TN];
};

// Shape of the staged tiles: rows of 128 bytes.
template <class C>
struct Stage8 {
    static constexpr int XSLOT = C::BM * kK8 / 16, WSLOT = C::BN * kK8 / 16;  // uint4
    static constexpr int XINS = XSLOT / 64 / C::NW, WINS = WSLOT / 64 / C::NW;  // loads per wave
    static_assert(XINS * 64 * C::NW == XSLOT && WINS * 64 * C::NW == WSLOT, "whole loads");
    // what the delta and the store stage fits
    static_assert(XSLOT >= 2 * C::XSLOT && WSLOT >= 2 * C::WSLOT, "two bf16 slots per slot");
};

__device__ __forceinline__ int swz8(int row) { return (row >> 1) & 7; }

// 32 codes of a row: chunks 4 h + g and 4 h + g + 2 (h: the step of the stage)
__device__ __forceinline__ i32x8_t read_row8(const uint4 *__restrict__ s, int row, int h, int g) {
    const int sw = swz8(row), c = 4 * h + g;
    const i32x4_t lo = *reinterpret_cast<const i32x4_t *>(&s[row * 8 + (c ^ sw)]);
    const i32x4_t hi = *reinterpret_cast<const i32x4_t *>(&s[row * 8 + ((c + 2) ^ sw)]);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

template <class C>
__device__ __forceinline__ void read_frags8(Frags8<C> &f, const uint4 *__restrict__ xs,
                                            const uint4 *__restrict__ ws, int h, int lane, int wm0,
                                            int wn0) {
    const int li = lane & 31, g = lane >> 5;
#pragma unroll
    for (int i = 0; i < C::TM; ++i) f.a[i] = read_row8(xs, wm0 + 32 * i + li, h, g);
#pragma unroll
    for (int j = 0; j < C::TN; ++j) f.b[j] = read_row8(ws, wn0 + 32 * j + li, h, g);
}

// WIDE: the codes widened to bf16, octet by octet.  INT: each of the lane's two chunks of every operand
// is one instruction's.
template <class C, bool WIDE, bool INT>
__device__ __forceinline__ void mfma_frags8(Sum8<INT> (&acc)[C::TM][C::TN], const Frags8<C> &f) {
    if constexpr (INT) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < C::TM; ++i)
#pragma unroll
                for (int j = 0; j < C::TN; ++j) {
                    const i32x4_t a = q == 0 ? __builtin_shufflevector(f.a[i], f.a[i], 0, 1, 2, 3)
                                             : __builtin_shufflevector(f.a[i], f.a[i], 4, 5, 6, 7);
                    const i32x4_t b = q == 0 ? __builtin_shufflevector(f.b[j], f.b[j], 0, 1, 2, 3)
                                             : __builtin_shufflevector(f.b[j], f.b[j], 4, 5, 6, 7);
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, acc[i][j], 0, 0, 0);
                }
        return;
    } else if constexpr (WIDE) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            bf16x8_t b[C::TN];
#pragma unroll
            for (int j = 0; j < C::TN; ++j)
                b[j] = __builtin_bit_cast(bf16x8_t, e4m3x8_to_bf16((uint32_t)f.b[j][2 * q],
                                                                   (uint32_t)f.b[j][2 * q + 1]));
#pragma unroll
            for (int i = 0; i < C::TM; ++i) {
                const bf16x8_t a = __builtin_bit_cast(
                    bf16x8_t, e4m3x8_to_bf16((uint32_t)f.a[i][2 * q], (uint32_t)f.a[i][2 * q + 1]));
#pragma unroll
                for (int j = 0; j < C::TN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b[j], acc[i][j], 0, 0, 0);
            }
        }
        return;
    } else {
#pragma unroll
        for (int i = 0; i < C::TM; ++i)
#pragma unroll
            for (int j = 0; j < C::TN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(f.a[i], f.b[j], acc[i][j], 0, 0,
                                                                            0, 0, 0, 0);
    }
}

// The next step's LDS reads among this step's MFMAs.
template <class C, bool INT>
__device__ __forceinline__ void interleave_reads8() {
    constexpr int reads = 2 * (C::TM + C::TN), mfmas = (INT ? 2 : 1) * C::TM * C::TN;
    constexpr int groups = mfmas < 4 ? mfmas : 4;
#pragma unroll
    for (int gi = 0; gi < groups; ++gi) {
        __builtin_amdgcn_sched_group_barrier(0x100, (reads + groups - 1) / groups, 0);  // DS reads
        __builtin_amdgcn_sched_group_barrier(0x008, mfmas / groups, 0);                 // MFMA
    }
}

// Direct-load sources of a lane, k = 0: load q of an operand covers tile rows 8 q .. 8 q + 7; lane
// i fills row 8 q + i / 8, stored chunk i % 8, which holds chunk (i % 8) ^ swz8(row).  As 32-bit
// byte offsets when both operands fit in 4 GiB (one VGPR per address).
template <class C>
struct Src8 {
    const uint8_t *xp[Stage8<C>::XINS], *wp[Stage8<C>::WINS];
    __device__ __forceinline__ const uint8_t *x(int j, int k0) const { return xp[j] + k0; }
    __device__ __forceinline__ const uint8_t *w(int j, int k0) const { return wp[j] + k0; }
};
template <class C>
struct Src8O32 {
    const uint8_t *xb, *wb;
    uint32_t xo[Stage8<C>::XINS], wo[Stage8<C>::WINS];
    __device__ __forceinline__ const uint8_t *x(int j, int k0) const { return xb + (uint32_t)(xo[j] + (uint32_t)k0); }
    __device__ __forceinline__ const uint8_t *w(int j, int k0) const { return wb + (uint32_t)(wo[j] + (uint32_t)k0); }
};

template <class C, class S>
__device__ __forceinline__ void issue8(const S &src, uint4 *__restrict__ xslot,
                                       uint4 *__restrict__ wslot, int wave, int k0) {
    constexpr int XI = Stage8<C>::XINS, WI = Stage8<C>::WINS;
#pragma unroll
    for (int j = 0; j < XI; ++j)
        __builtin_amdgcn_global_load_lds((const void *)src.x(j, k0),
                                         (lds_void_t *)&xslot[(wave * XI + j) * 64], 16, 0, 0);
#pragma unroll
    for (int j = 0; j < WI; ++j)
        __builtin_amdgcn_global_load_lds((const void *)src.w(j, k0),
                                         (lds_void_t *)&wslot[(wave * WI + j) * 64], 16, 0, 0);
}

// Register-path fill of a slot with rows r0 .. of an operand [rows][K], k0 .. k0 + 127 (zero
// beyond k1): the last stage where K is not a multiple of 128.
template <int ROWS, int NT>
__device__ __forceinline__ void fill8(uint4 *slot, const uint8_t *__restrict__ src, int rows,
                                      int K, int r0, int k0, int k1, const int32_t *perm, int tid) {
    for (int c = tid; c < ROWS * 8; c += NT) {
        const int row = c >> 3, lc = c & 7;
        const int rr = min(r0 + row, rows - 1);
        const int k = k0 + lc * 16;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (k < k1) v = ld16(src + (size_t)(perm ? perm[rr] : rr) * K + k);
        slot[row * 8 + (lc ^ swz8(row))] = v;
    }
}

// X: E4M3 codes (uint8_t) or integers (int8_t).  WIDE: y is fp32 (see the top).  FUSED: whole K, rows in segment order, delta and epilogue; else slice blockIdx.y of K, rows in
// their own order, into partial[blockIdx.y][M][N].
template <class C, class X, bool FUSED, bool WIDE, bool O32>
__global__ __launch_bounds__(C::NT, 2) void gemm_fp8_kernel(
    const X *__restrict__ x, const X *__restrict__ W,
    const float *__restrict__ w_scale, int M, int K, int N, int k_per_split,
    float *__restrict__ partial, void *y, int n_tm, int n_tn, Seg seg, LoraEpilogue ep,
    Epilogue epi) {
    using G = Stage8<C>;
    constexpr bool INT = std::is_same_v<X, int8_t>;
    const uint8_t *const x8 = reinterpret_cast<const uint8_t *>(x), *const W8 = reinterpret_cast<const uint8_t *>(W);
    __shared__ __attribute__((aligned(1024))) uint4 X0[G::XSLOT];
    __shared__ __attribute__((aligned(1024))) uint4 X1[G::XSLOT];
    __shared__ __attribute__((aligned(1024))) uint4 W0[G::WSLOT];
    __shared__ __attribute__((aligned(1024))) uint4 W1[G::WSLOT];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm0 = (wave / C::WN) * C::WTM, wn0 = (wave % C::WN) * C::WTN;
    int tmi, tni;
    tile_of(blockIdx.x, n_tm, n_tn, tmi, tni);
    const int row0 = tmi * C::BM, n0 = tni * C::BN;
    const int k_lo = FUSED ? 0 : (int)blockIdx.y * k_per_split;
    const int k_hi = FUSED ? K : min(K, k_lo + k_per_split);
    __shared__ RowTable<C> rows;
    const int my_row = FUSED ? seg.perm[min(row0 + tid, M - 1)] : 0;

    // rows beyond M and columns beyond N repeat the last one; their results are never stored
    std::conditional_t<O32, Src8O32<C>, Src8<C>> src;
    if constexpr (O32) {
        src.xb = x8;
        src.wb = W8;
    }
#pragma unroll
    for (int j = 0; j < G::XINS; ++j) {
        const int row = 8 * (wave * G::XINS + j) + (lane >> 3);
        const int rr = min(row0 + row, M - 1);
        const size_t o = (size_t)(FUSED ? seg.perm[rr] : rr) * K + ((lane & 7) ^ swz8(row)) * 16;
        if constexpr (O32) src.xo[j] = (uint32_t)o;
        else src.xp[j] = x8 + o;
    }
#pragma unroll
    for (int j = 0; j < G::WINS; ++j) {
        const int row = 8 * (wave * G::WINS + j) + (lane >> 3);
        const size_t o = (size_t)min(n0 + row, N - 1) * K + ((lane & 7) ^ swz8(row)) * 16;
        if constexpr (O32) src.wo[j] = (uint32_t)o;
        else src.wp[j] = W8 + o;
    }

    Sum8<INT> sum[C::TM][C::TN];
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
#pragma unroll
        for (int j = 0; j < C::TN; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) sum[i][j][v] = 0;

    // Per stage: multiply its first step while reading the second; then wait for the next
    // stage's loads (issued a stage ago) and, at the barrier, for every wave to have read this
    // slot; load the stage after next into it; multiply the second step while reading the next
    // stage's first.  Loads past the last stage reload it into a slot that is never multiplied.
    const int n = (k_hi - k_lo) / kK8;
    if (n > 0) {
        Frags8<C> fa, fb;
        issue8<C>(src, X0, W0, wave, k_lo);
        if constexpr (FUSED) fill_row<C>(rows, my_row, ep, seg, epi.row_scale, row0, tid);
        wait_vm<0>();
        lds_barrier();
        issue8<C>(src, X1, W1, wave, k_lo + min(1, n - 1) * kK8);
        if (FUSED && wave == C::NW - 1) fill_runs<C>(rows, lane);
        read_frags8<C>(fa, X0, W0, 0, lane, wm0, wn0);
#define LORA_FP8_STAGE(XP, WP, XQ, WQ)                                           \
        read_frags8<C>(fb, XP, WP, 1, lane, wm0, wn0);                           \
        mfma_frags8<C, WIDE, INT>(sum, fa);                                      \
        if constexpr (!WIDE || INT) interleave_reads8<C, INT>();                 \
        wait_vm<0>();                                                            \
        lds_barrier();                                                           \
        issue8<C>(src, XP, WP, wave, k_lo + min(s + 2, n - 1) * kK8);            \
        read_frags8<C>(fa, XQ, WQ, 0, lane, wm0, wn0);                           \
        mfma_frags8<C, WIDE, INT>(sum, fb);                                      \
        if constexpr (!WIDE || INT) interleave_reads8<C, INT>();                 \
        if (++s == n) break;
        for (int s = 0;;) {
            LORA_FP8_STAGE(X0, W0, X1, W1)
            LORA_FP8_STAGE(X1, W1, X0, W0)
        }
#undef LORA_FP8_STAGE
        wait_vm<0>();
    } else if constexpr (FUSED) {
        fill_row<C>(rows, my_row, ep, seg, epi.row_scale, row0, tid);
    }
    // the last stage, where it is partial: through registers, zero beyond k_hi
    if (const int k0 = k_lo + n * kK8; k0 < k_hi) {
        lds_barrier();
        if (FUSED && n == 0 && wave == C::NW - 1) fill_runs<C>(rows, lane);
        fill8<C::BM, C::NT>(X0, x8, M, K, row0, k0, k_hi, FUSED ? seg.perm : nullptr, tid);
        fill8<C::BN, C::NT>(W0, W8, N, K, n0, k0, k_hi, nullptr, tid);
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (k0 + 64 * h < k_hi) {
                Frags8<C> f;
                read_frags8<C>(f, X0, W0, h, lane, wm0, wn0);
                mfma_frags8<C, WIDE, INT>(sum, f);
            }
        }
    }

    // the columns' scales (an integer sum is rounded to fp32 here)
    f32x16_t acc[C::TM][C::TN];
#pragma unroll
    for (int j = 0; j < C::TN; ++j) {
        const float ws = w_scale[min(n0 + wn0 + 32 * j + (lane & 31), N - 1)];
#pragma unroll
        for (int i = 0; i < C::TM; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = (float)sum[i][j][v] * ws;
    }

    if constexpr (FUSED) {
        // (a stage's slot holds two of the bf16 steps')
        uint4 *const xs[4] = {X0, X0 + C::XSLOT, X1, X1 + C::XSLOT};
        uint4 *const ws[4] = {W0, W0 + C::WSLOT, W1, W1 + C::WSLOT};
        add_lora_runs<C, WIDE>(acc, xs, ws, ep, rows, M, N, n0, tid, lane, wm0, wn0);
        lds_barrier();
        // two waves per slot with eight waves, one with four
        constexpr int H = C::NW / 4;
        uint4 *const base = wave / H == 0 ? X0 : wave / H == 1 ? X1 : wave / H == 2 ? W0 : W1;
        uint4 *const sl = base + wave % H * (G::XSLOT / H);
        static_assert(G::XSLOT == G::WSLOT && G::XSLOT / H * 16 >= 16 * (C::WTN + 8) * 4, "staging fits");
        store_epilogue<C, WIDE>(acc, reinterpret_cast<float *>(sl), epi, y, rows, M, N, row0, wm0,
                                n0 + wn0, lane);
    } else {
        float *P = partial + (size_t)blockIdx.y * M * N;
#pragma unroll
        for (int i = 0; i < C::TM; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const int rr = row0 + wm0 + 32 * i + (v / 4) * 8 + (lane >> 5) * 4 + (v % 4);
                if (rr >= M) continue;
#pragma unroll
                for (int j = 0; j < C::TN; ++j) {
                    const int col = n0 + wn0 + 32 * j + (lane & 31);
                    if (col < N) P[(size_t)rr * N + col] = acc[i][j][v];
                }
            }
    }
}

template <class C, bool FUSED, class X>
hipError_t launch_fp8_cfg(const Gemm8<X> &g, const Fp8Plan &p, void *y, bool y_f32, Seg seg,
                          const LoraEpilogue &ep, const Epilogue &epi, float *partial,
                          hipStream_t s) {
    const int n_tm = (g.M + C::BM - 1) / C::BM, n_tn = (g.N + C::BN - 1) / C::BN;
    const bool o32 = (size_t)g.M * g.K <= 0xFFFFFFFFull && (size_t)g.N * g.K <= 0xFFFFFFFFull;
    const dim3 grid(n_tm * n_tn, p.ks);
#define FP8_ONE(WIDE, O32)                                                                     \
    launch((gemm_fp8_kernel<C, X, FUSED, WIDE, O32>), grid, dim3(C::NT), 0, s, g.x8, g.W8, g.w_scale, \
           g.M, g.K, g.N, p.k_per_split, partial, y, n_tm, n_tn, seg, ep, epi)
    if (y_f32 && C::BM != 128) return hipErrorInvalidValue;  // (fp8_plan: fp32 y takes the small tiles)
    // (slices of integers are the same for both types of y)
    if constexpr (C::BM == 128 && (FUSED || std::is_same_v<X, uint8_t>)) {
        if (y_f32) {
            if (o32) FP8_ONE(true, true);
            else FP8_ONE(true, false);
            return hipGetLastError();
        }
    }
    if (o32) FP8_ONE(false, true);
    else FP8_ONE(false, false);
#undef FP8_ONE
    return hipGetLastError();
}

}  // namespace

// A slice of K is a multiple of two stages.
constexpr int kMinK = 2 * kK8;

// Up to 256 small tiles may split K, into as many slices as two workgroups per CU hold at once. That
// costs the slices' way through memory and a launch (the more, the more tiles); whole tiles cost a
// walk through K at a workgroup or two per CU and, behind it, one through the adapter runs of the
// tile's rows, at every rank chunk (one slice is worth it for the latter alone).  us split and whole,
// d_out 4096: rank 16 of 4 adapters 520 x 1024 36.5 and 26.1, 520 x 4112 46.0 and 49.4, 520 x 11008
// 62.2 and 77.3, 1024 x 4112 59.6 and 54.2; rank 64 of 64 260 x 512 37.0 and 89.1, 1024 x 512 58.9 and 50.3
// (the rule takes the slices), 1024 x 4112 90.4 and 95.2; d_out 264, rank 16 of 4: 260 x 2048 27.1 and
// 27.2, 260 x 4112 28.7 and 36.2.  Rounds: 768 x 11008 x 4096 97 us in two slices, 118 in three (a second, short
// round).  Above 256 tiles the slices cost more than they bring: 1280 x 4096 x 4096 80 -> 88 us,
// 1536 x 11008 144 -> 164 with three.
Fp8Plan fp8_plan(int M, int K, int N, bool y_f32, int r_max, int n_adapters) {
    Fp8Plan p{};
    p.ks = 1;
    p.k_per_split = K;
    const long t128 = (long)((M + 127) / 128) * ((N + 127) / 128);
    const long runs = 128L * (n_adapters < M ? n_adapters : M) / (M > 128 ? M : 128);
    p.big = wide_tiles(M, N) && !y_f32;
    p.split = t128 <= 256 && K + 10L * r_max * runs > 2600 + 9 * t128;
    if (p.split) {
        const int steps = (K + kMinK - 1) / kMinK;
        int ks = (int)(512 / t128);  // two workgroups per CU, one round
        if (ks > 16) ks = 16;
        if (ks > steps) ks = steps;
        const int per = (steps + ks - 1) / ks;
        p.k_per_split = per * kMinK;
        p.ks = (K + p.k_per_split - 1) / p.k_per_split;
    }
    return p;
}

size_t fp8_partial_floats(int M, int K, int N, int r_max, int n_adapters) {
    // (the split does not depend on y's type)
    const Fp8Plan p = fp8_plan(M, K, N, true, r_max, n_adapters);
    return p.split ? (size_t)p.ks * M * N : 0;
}

template <class X>
hipError_t launch_gemm_fp8(const Gemm8<X> &g, const Fp8Plan &p, void *y, bool y_f32, Seg seg,
                           const LoraEpilogue &ep, const Epilogue &epi, float *partial,
                           hipStream_t s) {
    if (g.M < 1 || g.K < 16 || g.K % 16 != 0 || g.N < 8 || g.N % 8 != 0) return hipErrorInvalidValue;
    if (p.split) {
        if (partial == nullptr || p.k_per_split % kMinK != 0) return hipErrorInvalidValue;
        return launch_fp8_cfg<Big<128, 128>, false>(g, p, y, y_f32, seg, ep, epi, partial, s);
    }
    if (p.big) return launch_fp8_cfg<Big<256, 256, 2, 4>, true>(g, p, y, y_f32, seg, ep, epi, nullptr, s);
    return launch_fp8_cfg<Big<128, 128>, true>(g, p, y, y_f32, seg, ep, epi, nullptr, s);
}
template hipError_t launch_gemm_fp8(const Gemm8<uint8_t> &, const Fp8Plan &, void *, bool, Seg,
                                    const LoraEpilogue &, const Epilogue &, float *, hipStream_t);
template hipError_t launch_gemm_fp8(const Gemm8<int8_t> &, const Fp8Plan &, void *, bool, Seg,
                                    const LoraEpilogue &, const Epilogue &, float *, hipStream_t);

}  // namespace lora
