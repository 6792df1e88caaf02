// big_tiles.h -- what the large-tile MFMA GEMMs share (csrc/gemm_big.hip on bf16, csrc/gemm_fp8.hip
// on 8-bit operands): tile shapes, waits, the bf16 operand fragments of one 32-deep step, the
// LoRA delta added as extra MFMA steps after the K loop, and the store with an epilogue.
#pragma once

#include "epilogue.h"

namespace lora {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void_t;
typedef __attribute__((address_space(3))) bf16x4_t lds_bf16x4_t;
typedef __attribute__((address_space(3))) char lds_char_t;

constexpr int kBK = 32;     // k per stage

// Tile BM x BN computed by WM x WN waves, each owning (BM / WM) x (BN / WN).
template <int BM_, int BN_, int WM_ = 2, int WN_ = 2>
struct Big {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr int NW = WM * WN, NT = 64 * NW;  // waves, threads
    static constexpr int WTM = BM / WM, WTN = BN / WN;  // per-wave tile
    static constexpr int TM = WTM / 32, TN = WTN / 32;
    static constexpr int XSLOT = BM * kBK * 2 / 16;  // uint4 per x slot
    static constexpr int WSLOT = kBK * BN * 2 / 16;  // uint4 per W slot
    static constexpr int XINS = XSLOT / 64 / NW;     // DMA instructions per wave per stage
    static constexpr int WINS = WSLOT / 64 / NW;
    static constexpr int PER = XINS + WINS;
    static constexpr int WROWS = 1024 / (BN * 2);     // W rows per DMA instruction
    static constexpr int WCH = BN / 8;                // 16-byte chunks per W row
    static_assert(BN == 128 || BN == 256, "W swizzle needs at least 16 chunks per row");
    static_assert(BM == 128 || BM == 256, "x tile");
    static_assert(XINS >= 1 && WINS >= 1, "per-wave DMA split");
    static_assert(XINS * 64 * NW == XSLOT && WINS * 64 * NW == WSLOT, "whole DMA instructions");
    static_assert(NW == 4 || NW == 8, "four or eight waves (staging slots)");
    static_assert(TM >= 1 && TN >= 1, "per-wave tile of whole 32 x 32 blocks");
};

// s_waitcnt with only vmcnt = n (n < 64); expcnt and lgkmcnt left at their maxima.
template <int N>
__device__ __forceinline__ void wait_vm() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
}

// Workgroup barrier that orders LDS accesses in the compiler but adds no vmcnt wait.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's LDS reads have returned
    asm volatile("s_barrier" ::: "memory");
}

// ---- operand fragments of one 32-deep step ------------------------------------------------
// a[kk][i]: rows wm0 + 32 i + lane % 32, k = 16 kk + 8 (lane / 32) .. +7 (one ds_read_b128);
// b[kk][j]: column wn0 + 32 j + lane % 32, the same 8 k (two ds_read_b64_tr_b16).
template <class C>
struct Frags {
    bf16x8_t a[2][C::TM];
    bf16x8_t b[2][C::TN];
};

template <class C>
__device__ __forceinline__ void read_frags(Frags<C> &f, const uint4 *__restrict__ xs,
                                           const uint4 *__restrict__ ws, int lane, int wm0,
                                           int wn0) {
    const lds_char_t *wsb = (const lds_char_t *)(ws);
    const int g = lane >> 4, li = lane & 15;
    const int rsw = (li >> 2) << 2;  // (row % 4) * 4 for every W row this lane names
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
        for (int i = 0; i < C::TM; ++i) {
            const int row = wm0 + 32 * i + (lane & 31);
            const int lc = 2 * kk + (lane >> 5);
            f.a[kk][i] = *reinterpret_cast<const bf16x8_t *>(&xs[row * 4 + (lc ^ ((row >> 2) & 3))]);
        }
#pragma unroll
        for (int j = 0; j < C::TN; ++j) {
            const int col = wn0 + 32 * j + 16 * (g & 1) + 4 * (li & 3);
            const int lc = col >> 3, half = (col >> 2) & 1;
            const int r = 16 * kk + 8 * (g >> 1) + (li >> 2);
            const lds_char_t *p = wsb + r * (C::BN * 2) + ((lc ^ rsw) << 4) + half * 8;
            const bf16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4_t *)p);
            const bf16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4_t *)(p + 4 * C::BN * 2));
            f.b[kk][j] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
}

template <class C>
__device__ __forceinline__ void mfma_frags(f32x16_t (&acc)[C::TM][C::TN], const Frags<C> &f) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int i = 0; i < C::TM; ++i)
#pragma unroll
            for (int j = 0; j < C::TN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[kk][i], f.b[kk][j], acc[i][j], 0, 0, 0);
}

// One 32-deep step straight from LDS (used outside the pipelined loop).
template <class C>
__device__ __forceinline__ void mfma_stage(f32x16_t (&acc)[C::TM][C::TN],
                                           const uint4 *__restrict__ xs,
                                           const uint4 *__restrict__ ws, int lane, int wm0, int wn0) {
    Frags<C> f;
    read_frags<C>(f, xs, ws, lane, wm0, wn0);
    mfma_frags<C>(acc, f);
}

// Interleave the LDS reads of the next step's fragments with this step's MFMAs: groups of
// DS reads, then MFMAs, in order (one scheduling group sequence).
template <class C>
__device__ __forceinline__ void interleave_reads_with_mfma() {
    constexpr int reads = 2 * (C::TM + 2 * C::TN);
    constexpr int mfmas = 2 * C::TM * C::TN;
    constexpr int groups = 8;
    constexpr int rpg = (reads + groups - 1) / groups;
    constexpr int mpg = mfmas / groups;
#pragma unroll
    for (int gi = 0; gi < groups; ++gi) {
        __builtin_amdgcn_sched_group_barrier(0x100, rpg, 0);  // DS reads
        __builtin_amdgcn_sched_group_barrier(0x008, mpg, 0);  // MFMA
    }
}

// Tile order: XCD-major (workgroup b runs on XCD b % 8), then groups of 4 tile rows, column-
// major inside a group, so each XCD works on a compact block of tiles.
__device__ __forceinline__ void tile_of(int b, int n_tm, int n_tn, int &tm, int &tn) {
    const int T = n_tm * n_tn;
    int lin = b;
    if ((T % 8) == 0) lin = (b % 8) * (T / 8) + b / 8;
    constexpr int G = 4;
    const int group = lin / (G * n_tn);
    const int first = group * G;
    const int gsz = min(n_tm - first, G);
    const int in = lin % (G * n_tn);
    tm = first + in % gsz;
    tn = in / gsz;
}

// What the end of a tile needs of its rows (positions of perm), read once at its start, in the
// shadow of the first stage's loads: a chain perm -> ids, row scale per step of the store cost a
// prefill tile more than its MFMAs' last third.
template <class C>
struct RowTable {
    int32_t m[C::BM];    // row of x and y (rows past the last repeat it)
    int32_t id[C::BM];   // its adapter
    float scale[C::BM];  // its x scale (1 without)
};

// Thread tid fills row tid, whose row of x is m (read before the first stage's loads are
// issued; this follows them).  A barrier must come before the table is read.
template <class C>
__device__ __forceinline__ void fill_row(RowTable<C> &t, int m, const int32_t *ids,
                                         const float *row_scale, int tid) {
    static_assert(C::NT >= C::BM, "one row per thread");
    if (tid < C::BM) {
        t.m[tid] = m;
        t.id[tid] = ids[m];
        t.scale[tid] = row_scale ? row_scale[m] : 1.0f;
    }
}

// The LoRA delta of one output tile (rows in segment order), after its K loop: acc += scale_a
// t[rows, :] B_a[:, columns] for every run of one adapter among the tile's rows.  X0 and W0 are
// LDS slots free for staging once every wave has passed the first barrier here.
//
// Runs of one adapter among this tile's rows (positions of perm): for each run, 16
// rank columns at a time, stage T = scale_a * t[rows, :] (zero outside the run) in
// slot 0's x layout as a pair of bf16 values per element -- k slots 0..15 the value
// rounded to bf16, slots 16..31 the remainder (exact in fp32) rounded to bf16 -- and
// B_a's same 16 rank rows twice in its W layout (zero beyond the rank), then one more
// MFMA step.  The pair carries scale * t to about 16 significant bits, so the delta is
// not rounded to bf16 precision before it is added.
template <class C>
__device__ __forceinline__ void add_lora_runs(f32x16_t (&acc)[C::TM][C::TN], uint4 *X0, uint4 *W0,
                                              const LoraEpilogue &ep, const Seg &seg,
                                              const RowTable<C> &rows, int M, int N, int row0,
                                              int n0, int tid, int lane, int wm0, int wn0) {
    const int n_lora = seg.meta[1];
    const int RM = ep.r_max;
    constexpr int kHalf = kBK / 2;
    int p = row0;
    const int p_end = min(row0 + C::BM, n_lora);
    while (p < p_end) {
        const int a = rows.id[p - row0];
        if (a < 0 || a >= ep.n_adapters) break;  // segments not built for these ids
        const int q_end = min(seg.offsets[a + 1], p_end);
        if (q_end <= p) break;
        const float s = ep.scale[a];
        // B_a's rank rows: all of a padded pool's stride (zero past the rank), the
        // rank's in a compact one
        int ra = ep.roff ? min(max(ep.ranks[a], 0), RM) : ep.pstride;
        const int brow0 = adapter_row0(ep.roff, ep.pool_rows, a, ep.pstride, ra);
        for (int rc = 0; rc < RM; rc += kHalf) {
            lds_barrier();
            for (int c = tid; c < C::BM * 4; c += C::NT) {
                const int row = c >> 2, lc = c & 3;
                const int pos = row0 + row;
                const int j = rc + (lc & 1) * 8;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (pos >= p && pos < q_end && j < RM) {
                    // t[m, j .. j+7]: the shrink's chunk sums added in chunk order, four
                    // chunks' loads in flight at a time
                    const float *tp = ep.tpart + (size_t)rows.m[row] * RM + j;
                    const size_t cs = (size_t)M * RM;
                    float t[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                    for (int c0 = 0; c0 < ep.n_chunks; c0 += 4) {
                        float4 v[4][2];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const bool in = c0 + c < ep.n_chunks;
                            const float *q = tp + (size_t)(in ? c0 + c : 0) * cs;
                            v[c][0] = in ? *reinterpret_cast<const float4 *>(q) : make_float4(0.f, 0.f, 0.f, 0.f);
                            v[c][1] = in ? *reinterpret_cast<const float4 *>(q + 4) : make_float4(0.f, 0.f, 0.f, 0.f);
                        }
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            if (c0 + c < ep.n_chunks) {
                                t[0] += v[c][0].x; t[1] += v[c][0].y; t[2] += v[c][0].z; t[3] += v[c][0].w;
                                t[4] += v[c][1].x; t[5] += v[c][1].y; t[6] += v[c][1].z; t[7] += v[c][1].w;
                            }
                        }
                    }
                    float f[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = s * t[e];
                    if (lc >= 2) {  // the remainder after rounding to bf16
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] -= __uint_as_float(f32_to_bf16_rne(f[e]) << 16);
                    }
                    v = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                   pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
                }
                X0[row * 4 + (lc ^ ((row >> 2) & 3))] = v;
            }
            for (int c = tid; c < kBK * C::WCH; c += C::NT) {
                const int r = c / C::WCH, lc = c % C::WCH;
                const int rank = rc + (r & (kHalf - 1));
                const int n = n0 + lc * 8;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (rank < ra && n < N) v = ld16(ep.B + ((size_t)brow0 + rank) * N + n);
                W0[r * C::WCH + (lc ^ ((r & 3) << 2))] = v;
            }
            __syncthreads();
            mfma_stage<C>(acc, X0, W0, lane, wm0, wn0);
        }
        p = q_end;
    }
}

// Stores a wave's WTM x WTN block of the tile (first position row0 + wm0, first column c0) with
// the epilogue.  It stages 16 fp32 rows at a time in its own LDS slot stg, so that a lane then holds
// 8 consecutive columns of a row: mul, residual and y move in 16-byte pieces.  mul and residual
// are loaded AHEAD steps before their use (what the accumulators leave of the registers).  bf16 y
// is stored nontemporally, so that the end of the kernel finds fewer dirty lines in the L2s (fp8
// 4096 x 4096 x 4096: 72.5 -> 69.4 us, 4096 x 4096 x 11008 without gate: 210 -> 193 us).  LDS
// accesses of one wave complete in order, so the staging needs no barrier beyond the one that
// freed the slots.
template <class C, bool YF32>
__device__ __forceinline__ void store_epilogue(const f32x16_t (&acc)[C::TM][C::TN], float *stg,
                                               const Epilogue &epi, void *y,
                                               const RowTable<C> &rows, int M, int N, int row0,
                                               int wm0, int c0, int lane) {
    constexpr int SROW = C::WTN + 8;   // staged row length (floats): 4 rows apart, 32 banks apart
    constexpr int CPR = C::WTN / 8;    // 8-column pieces per row
    constexpr int PP = 16 * CPR / 64;  // pieces per lane and step
    constexpr int STEPS = 2 * C::TM;
    constexpr int AHEAD = YF32 ? 1 : 3;
    static_assert(16 * SROW * 4 <= C::XSLOT * 16 && 16 * SROW * 4 <= C::WSLOT * 16,
                  "staging fits one slot");
    static_assert(PP * 64 == 16 * CPR, "whole pieces");
    EpiOperands<8, YF32> eo[AHEAD + 1][PP];
    const int pr = lane / CPR, pc = 8 * (lane % CPR);  // this lane's row (of 64 / CPR) and column
    const int col = c0 + pc, colc = min(col, N - 8);
    EpiOperands<8, YF32> fixed;
    fixed.load_bias(epi, colc);
    auto row_of = [&](int st, int q) { return wm0 + 16 * st + pr + q * (64 / CPR); };
    auto operands = [&](int st) {
#pragma unroll
        for (int q = 0; q < PP; ++q) eo[st % (AHEAD + 1)][q].load_row(epi, rows.m[row_of(st, q)], colc, N);
    };
#pragma unroll
    for (int st = 0; st < AHEAD; ++st) operands(st);
#pragma unroll
    for (int st = 0; st < STEPS; ++st) {
        const int i = st >> 1, h = st & 1;
        if (st + AHEAD < STEPS) operands(st + AHEAD);
#pragma unroll
        for (int j = 0; j < C::TN; ++j)
#pragma unroll
            for (int v = 0; v < 8; ++v)
                stg[((v / 4) * 8 + (lane >> 5) * 4 + (v % 4)) * SROW + 32 * j + (lane & 31)] =
                    acc[i][j][8 * h + v];
#pragma unroll
        for (int q = 0; q < PP; ++q) {
            const float *sp = &stg[(pr + q * (64 / CPR)) * SROW + pc];
            const float4 a = *reinterpret_cast<const float4 *>(sp);
            const float4 b = *reinterpret_cast<const float4 *>(sp + 4);
            float z[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            const int lr = row_of(st, q);
            EpiOperands<8, YF32> &o = eo[st % (AHEAD + 1)][q];
#pragma unroll
            for (int w = 0; w < 4; ++w) o.b[w] = fixed.b[w];
            o.rs = rows.scale[lr];
            o.apply(epi, z);
            if (row0 + lr < M && col < N) {
                const size_t at = (size_t)rows.m[lr] * N + col;
                if constexpr (YF32) {
                    float4 *yf = reinterpret_cast<float4 *>(reinterpret_cast<float *>(y) + at);
                    yf[0] = make_float4(z[0], z[1], z[2], z[3]);
                    yf[1] = make_float4(z[4], z[5], z[6], z[7]);
                } else {
                    st16_nt(reinterpret_cast<uint16_t *>(y) + at,
                            make_uint4(cvt_bf16x2(z[0], z[1]), cvt_bf16x2(z[2], z[3]),
                                       cvt_bf16x2(z[4], z[5]), cvt_bf16x2(z[6], z[7])));
                }
            }
        }
    }
}

}  // namespace

}  // namespace lora
