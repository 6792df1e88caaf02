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
__device__ __forceinline__ bf16x8_t read_a(const uint4 *__restrict__ xs, int kk, int i, int lane, int wm0) {
    const int row = wm0 + 32 * i + (lane & 31);
    const int lc = 2 * kk + (lane >> 5);
    return *reinterpret_cast<const bf16x8_t *>(&xs[row * 4 + (lc ^ ((row >> 2) & 3))]);
}
template <class C>
__device__ __forceinline__ bf16x8_t read_b(const uint4 *__restrict__ ws, int kk, int j, int lane, int wn0) {
    const lds_char_t *wsb = (const lds_char_t *)(ws);
    const int g = lane >> 4, li = lane & 15;
    const int rsw = (li >> 2) << 2;  // (row % 4) * 4 for every W row this lane names
    const int col = wn0 + 32 * j + 16 * (g & 1) + 4 * (li & 3);
    const int lc = col >> 3, half = (col >> 2) & 1;
    const int r = 16 * kk + 8 * (g >> 1) + (li >> 2);
    const lds_char_t *p = wsb + r * (C::BN * 2) + ((lc ^ rsw) << 4) + half * 8;
    const bf16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4_t *)p);
    const bf16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4_t *)(p + 4 * C::BN * 2));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}
template <class C>
__device__ __forceinline__ void read_frags(Frags<C> &f, const uint4 *__restrict__ xs,
                                           const uint4 *__restrict__ ws, int lane, int wm0,
                                           int wn0) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
        for (int i = 0; i < C::TM; ++i) f.a[kk][i] = read_a<C>(xs, kk, i, lane, wm0);
#pragma unroll
        for (int j = 0; j < C::TN; ++j) f.b[kk][j] = read_b<C>(ws, kk, j, lane, wn0);
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
// shadow of the first stage's loads: a chain perm -> ids -> ... at every step of the delta and the
// store took longer than their bytes do.
template <class C>
struct RowTable {
    int32_t m[C::BM];        // row of x and y (rows past the last repeat it)
    int32_t id[C::BM];       // its adapter, -1 without one
    float lora[C::BM];       // the adapter's scale
    float scale[C::BM];      // the row's x scale (1 without)
    int32_t run[C::BM + 1];  // first row of each run of one adapter, then BM
    int32_t n_runs;
};

// Thread tid fills row tid, whose row of x is m (read before the first stage's loads are
// issued; this follows them).  A barrier must come before the table is read.
template <class C>
__device__ __forceinline__ void fill_row(RowTable<C> &t, int m, const LoraEpilogue &ep, const Seg &seg,
                                         const float *row_scale, int row0, int tid) {
    static_assert(C::NT >= C::BM, "one row per thread");
    if (tid < C::BM) {
        // (positions at or past the LoRA row count, and ids outside the pool -- segments not built
        // for these ids -- have no t)
        const int id = ep.ids[m];
        const bool has = row0 + tid < seg.meta[1] && id >= 0 && id < ep.n_adapters;
        t.m[tid] = m;
        t.id[tid] = has ? id : -1;
        t.lora[tid] = has ? ep.scale[id] : 0.0f;
        t.scale[tid] = row_scale ? row_scale[m] : 1.0f;
    }
}

// The runs of the table's rows, by one wave behind the barrier that completes the table (the K loop's
// barriers then lie before their use).
template <class C>
__device__ __forceinline__ void fill_runs(RowTable<C> &t, int lane) {
    int n = 0;
#pragma unroll
    for (int r0 = 0; r0 < C::BM; r0 += 64) {
        const int r = r0 + lane;
        const bool first = r == 0 || t.id[r] != t.id[r - 1];
        const uint64_t mask = __ballot(first);
        if (first) t.run[n + __popcll(mask & ((1ull << lane) - 1))] = r;
        n += __popcll(mask);
    }
    if (lane == 0) {
        t.run[n] = C::BM;
        t.n_runs = n;
    }
}

// T's third part (EXACT) of a rank chunk: 16 k of every tile row, in the second half of a W slot
// (whose first half holds a step's 16 rows of B).  Chunk c of row r lies at c ^ ((r / 8) % 2), so that
// 16 rows of one chunk meet all banks once.
template <class C>
__device__ __forceinline__ uint4 *t3_of(uint4 *ws) {
    static_assert(kBK / 2 * C::WCH >= 2 * C::BM, "T's third part fits half a W slot");
    return ws + kBK / 2 * C::WCH;
}
__device__ __forceinline__ int t3_at(int row, int c) { return 2 * row + (c ^ ((row >> 3) & 1)); }

// 8 bf16 values -> -1, 0 or 1 by their sign, a NaN kept
__device__ __forceinline__ bf16x8_t signs8(bf16x8_t v) {
    const uint4 u = __builtin_bit_cast(uint4, v);
    uint32_t d[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint32_t o = 0;
#pragma unroll
        for (int s = 0; s < 32; s += 16) {
            const uint32_t h = (d[e] >> s) & 0xFFFFu, m = h & 0x7FFFu;
            o |= (m == 0 ? 0u : m > 0x7F80u ? h : (h & 0x8000u) | 0x3F80u) << s;
        }
        d[e] = o;
    }
    return __builtin_bit_cast(bf16x8_t, make_uint4(d[0], d[1], d[2], d[3]));
}

// Two bf16 values: infinities and NaN alone, others zeros (ODD), or the others alone, an infinity
// as 1 of its sign.
template <bool ODD>
__device__ __forceinline__ uint32_t odd_bf16x2(uint32_t d) {
    uint32_t o = 0;
#pragma unroll
    for (int s = 0; s < 32; s += 16) {
        const uint32_t h = (d >> s) & 0xFFFFu, m = h & 0x7FFFu;
        o |= (ODD ? (m >= 0x7F80u ? h : 0u)
                  : m < 0x7F80u ? h : m == 0x7F80u ? (h & 0x8000u) | 0x3F80u : 0u) << s;
    }
    return o;
}

// One bf16 step of the delta (T's parts, 16 k each, times the same 16 rows of B): T (xs, t3) holds every
// row's own, so rows outside lo <= row < hi (tile rows) are taken as zeros.  BY_ROW (the pass over
// infinities and NaN): T is its sign alone, and the products are added to the rows inside alone, so
// that 0 x infinity and 0 x NaN reach no other row.
template <class C, bool BY_ROW, bool EXACT>
__device__ __forceinline__ void mfma_run(f32x16_t (&acc)[C::TM][C::TN], const uint4 *__restrict__ xs,
                                         const uint4 *t3, const uint4 *ws, int lane, int wm0, int wn0,
                                         int lo, int hi) {
    constexpr int PARTS = BY_ROW ? 1 : EXACT ? 3 : 2;
    bf16x8_t b[C::TN];
#pragma unroll
    for (int j = 0; j < C::TN; ++j) b[j] = read_b<C>(ws, 0, j, lane, wn0);
#pragma unroll
    for (int i = 0; i < C::TM; ++i) {
        const int r0 = wm0 + 32 * i, row = r0 + (lane & 31);
        if (hi <= r0 || lo >= r0 + 32) continue;  // uniform: a block without a row of the run
        bf16x8_t a[PARTS];
#pragma unroll
        for (int kk = 0; kk < min(PARTS, 2); ++kk) a[kk] = read_a<C>(xs, kk, i, lane, wm0);
        if constexpr (BY_ROW) a[0] = signs8(a[0]);
        if constexpr (PARTS == 3) a[2] = *reinterpret_cast<const bf16x8_t *>(&t3[t3_at(row, lane >> 5)]);
#pragma unroll
        for (int kk = 0; kk < PARTS; ++kk)
            if (row < lo || row >= hi) a[kk] = __builtin_bit_cast(bf16x8_t, make_uint4(0, 0, 0, 0));
#pragma unroll
        for (int j = 0; j < C::TN; ++j) {
            if constexpr (BY_ROW) {
                f32x16_t p;
#pragma unroll
                for (int v = 0; v < 16; ++v) p[v] = 0.0f;
#pragma unroll
                for (int kk = 0; kk < PARTS; ++kk)
                    p = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[kk], b[j], p, 0, 0, 0);
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    const int rv = r0 + (v / 4) * 8 + (lane >> 5) * 4 + (v % 4);
                    acc[i][j][v] = rv >= lo && rv < hi ? acc[i][j][v] + p[v] : acc[i][j][v];
                }
            } else {
#pragma unroll
                for (int kk = 0; kk < PARTS; ++kk)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[kk], b[j], acc[i][j], 0, 0, 0);
            }
        }
    }
}

__device__ __forceinline__ uint4 bf16_parts8(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = bf16_part(f[2 * e]) | (bf16_part(f[2 * e + 1]) << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// T = scale_a * t of the tile's rows, every row with its own adapter: rank chunk q (16 columns) in
// slot q's x layout, as a pair of bf16 values per element -- k slots 0..15 the value rounded to
// bf16, slots 16..31 the remainder (exact in fp32) rounded to bf16.  The pair carries scale * t to
// about 16 significant bits, so the delta is not rounded to bf16 precision before it is added.  EXACT
// (fp32 y): what the pair leaves, again rounded to bf16, in W slot q's second half: the three carry
// all 24 bits.
template <class C, bool EXACT>
__device__ __forceinline__ void stage_t(uint4 *const (&xs)[4], uint4 *const (&ws)[4],
                                        const LoraEpilogue &ep, const RowTable<C> &rows, int M, int tid) {
    constexpr int kHalf = kBK / 2;
    const int RM = ep.r_max;
#pragma unroll 1
    for (int q = 0; q * kHalf < RM; ++q) {
        uint4 *const X = q == 0 ? xs[0] : q == 1 ? xs[1] : q == 2 ? xs[2] : xs[3];
        uint4 *const T3 = t3_of<C>(q == 0 ? ws[0] : q == 1 ? ws[1] : q == 2 ? ws[2] : ws[3]);
#pragma unroll 2
        for (int c = tid; c < C::BM * 4; c += C::NT) {
            const int row = c >> 2, lc = c & 3;
            const int j = q * kHalf + (lc & 1) * 8;
            uint4 v = make_uint4(0, 0, 0, 0), v3 = v;
            if (rows.id[row] >= 0 && j < RM) {
                // t[m, j .. j+7]: the shrink's chunk sums added in chunk order, four chunks'
                // loads in flight at a time
                const float *tp = ep.tpart + (size_t)rows.m[row] * RM + j;
                const size_t cs = (size_t)M * RM;
                float t[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                for (int c0 = 0; c0 < ep.n_chunks; c0 += 4) {
                    float4 p[4][2];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const bool in = c0 + k < ep.n_chunks;
                        const float *src = tp + (size_t)(in ? c0 + k : 0) * cs;
                        p[k][0] = in ? *reinterpret_cast<const float4 *>(src) : make_float4(0.f, 0.f, 0.f, 0.f);
                        p[k][1] = in ? *reinterpret_cast<const float4 *>(src + 4) : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (c0 + k < ep.n_chunks) {
                            t[0] += p[k][0].x; t[1] += p[k][0].y; t[2] += p[k][0].z; t[3] += p[k][0].w;
                            t[4] += p[k][1].x; t[5] += p[k][1].y; t[6] += p[k][1].z; t[7] += p[k][1].w;
                        }
                    }
                }
                const float s = rows.lora[row];
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = s * t[e];
                if (lc >= 2) {  // the remainder after rounding to bf16
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = bf16_rest(f[e]);
                }
                v = bf16_parts8(f);
                if (EXACT && lc >= 2) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = bf16_rest(f[e]);
                    v3 = bf16_parts8(f);
                }
            }
            X[row * 4 + (lc ^ ((row >> 2) & 3))] = v;
            if (EXACT && lc >= 2) T3[t3_at(row, lc & 1)] = v3;
        }
    }
}

// acc += T B_a for every run of one adapter among the tile's rows, in steps of 16 rank columns:
// B_a's 16 rank rows (for each of T's parts) in the first half of a W slot.  Four steps share their two barriers and
// have their loads in flight together, a batch ahead of their use (two more batches ahead changed
// nothing).  Waves, and 32-row blocks, without a row of a run skip its step.
//
// A row outside a run still meets the run's B, times zero.  So that an adapter whose B holds an
// infinity or a NaN spoils its own rows alone, a second pass (ODD, only when there are any) stages
// them alone, against the sign of T, and adds their products by rows: T of several parts, whose
// signs may differ, would make NaN of an infinite product.  Here such an infinity stands as 1 of its
// sign (an infinite T keeps its own) and a NaN as 0.  Returns whether there were any.
template <class C, bool ODD, bool EXACT>
__device__ __forceinline__ bool add_lora_steps(f32x16_t (&acc)[C::TM][C::TN], uint4 *const (&xs)[4],
                                               uint4 *const (&ws)[4], const LoraEpilogue &ep,
                                               const RowTable<C> &rows, int M, int N, int n0,
                                               int tid, int lane, int wm0, int wn0) {
    constexpr int kHalf = kBK / 2;
    const int RM = ep.r_max;
    const int sh = RM <= 16 ? 0 : RM == 32 ? 1 : 2;  // 2^sh rank chunks per run
    auto slot = [](int u, uint4 *const (&v)[4]) { return u == 0 ? v[0] : u == 1 ? v[1] : u == 2 ? v[2] : v[3]; };
    const int n_runs = __builtin_amdgcn_readfirstlane(rows.n_runs);
    wm0 = __builtin_amdgcn_readfirstlane(wm0);
    static_assert(kHalf * C::WCH == C::NT, "one piece of B per thread and step");
    const int br = tid / C::WCH, bc = tid % C::WCH, n = n0 + bc * 8;
    uint4 bv[4];
    // Step t of the tile: the runs are taken in two halves in turn, whose rows mostly belong to
    // different waves (in run order, half of the waves waited at each barrier for the other:
    // 1024 x 1024 x 4096 of 256 adapters rank 64, 131 -> 111 us; 256 x 256 tiles spill over it, 4096 x
    // 4096 x 4096 244 -> 262); a row meets its own run's rank chunks in ascending order.
    constexpr bool SIDES = C::BM == 128;
    const int two = SIDES && n_runs > 1 ? 1 : 0, half = two ? (n_runs + 1) / 2 : n_runs;
    const int n_steps = half << (sh + two);
    auto chunk_of = [&](int T0, int u) { return (SIDES && two ? (T0 + u) >> 1 : u) & ((1 << sh) - 1); };
    // Lane l holds the first row (SIDES: and the end) and the adapter of step T0 + l's run (else:
    // of the l-th run of the batch), which the steps take from there as scalars (read from LDS
    // step by step, they were a chain of two reads in front of each: 154 -> 131 us).
    int span, adapter;
    auto runs_of = [&](int T0) {
        if constexpr (SIDES) {
            const int t = T0 + lane, run = (t & two) * half + (t >> (sh + two));
            const int first = rows.run[min(run, n_runs)];
            span = first | rows.run[min(run + 1, n_runs)] << 16;
            adapter = t < n_steps && run < n_runs ? rows.id[first] : -1;
        } else {
            const int run = (T0 >> sh) + lane;
            span = rows.run[min(run, n_runs)];
            adapter = run < n_runs ? rows.id[span] : -1;
        }
    };
    auto lane_of = [&](int u) { return SIDES ? u : u >> sh; };
    // B_a's rank rows: all of a padded pool's stride (zero past the rank), the rank's in a
    // compact one
    auto load = [&](int T0) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int a = __builtin_amdgcn_readlane(adapter, lane_of(u));
            const int rank = chunk_of(T0, u) * kHalf + br;
            bv[u] = make_uint4(0, 0, 0, 0);
            if (a >= 0) {
                int ra = ep.roff ? min(max(ep.ranks[a], 0), RM) : ep.pstride;
                const int brow0 = adapter_row0(ep.roff, ep.pool_rows, a, ep.pstride, ra);
                if (rank < ra && n < N) bv[u] = ld16(ep.B + ((size_t)brow0 + rank) * N + n);
            }
        }
    };
    bool odd = false;
    runs_of(0);
    load(0);
    if constexpr (!ODD) stage_t<C, EXACT>(xs, ws, ep, rows, M, tid);  // (the first batch's barrier covers T too)
#pragma unroll 1
    for (int T0 = 0; T0 < n_steps; T0 += 4) {
        if (ODD || T0 > 0) lds_barrier();  // every wave is done with the W slots
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            uint32_t d[4] = {bv[u].x, bv[u].y, bv[u].z, bv[u].w};
            // an exponent of all ones, plus one, carries into its half's sign bit
            uint32_t ones = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) ones |= (d[e] & 0x7F807F80u) + 0x00800080u;
            if (ODD || (ones & 0x80008000u)) {
                odd = true;
#pragma unroll
                for (int e = 0; e < 4; ++e) d[e] = odd_bf16x2<ODD>(d[e]);
            }
            ws[u][br * C::WCH + (bc ^ ((br & 3) << 2))] = make_uint4(d[0], d[1], d[2], d[3]);
        }
        lds_barrier();
        const int rows_of = span, of = adapter;  // this batch's
        runs_of(T0 + 4);
        load(T0 + 4);
#pragma unroll 1
        for (int u = 0; u < 4; ++u) {
            const int k = lane_of(u), span_k = __builtin_amdgcn_readlane(rows_of, k);
            const int lo = SIDES ? span_k & 0xFFFF : span_k;
            const int hi = SIDES ? span_k >> 16 : __builtin_amdgcn_readlane(rows_of, k + 1);
            if (__builtin_amdgcn_readlane(of, k) < 0 || hi <= wm0 || lo >= wm0 + C::WTM) continue;  // uniform
            const int q = chunk_of(T0, u);
            mfma_run<C, ODD, EXACT>(acc, slot(q, xs), t3_of<C>(slot(q, ws)), slot(u, ws), lane, wm0, wn0, lo, hi);
        }
    }
    return __syncthreads_or(odd);
}

// The LoRA delta of one output tile (rows in segment order), after its K loop: acc += scale_a
// t[rows, :] B_a[:, columns].  xs, ws: four slot pairs, free once every wave has passed the first
// barrier here.  Whole call, 1, 8, 64 and 256 adapters of rank 16, us: 4096 x 4096 x 11008 8-bit rows
// 207, 209, 217, 251 (17 runs per tile in the last; the kernel alone 298 before T was staged once
// for every row and B loaded ahead); 4096 x 4096 x 4096 bf16 145, 145, 150, 162; 1300 x 1024 x 4096
// bf16 39, 39, 42, 54.
template <class C, bool EXACT>
__device__ __forceinline__ void add_lora_runs(f32x16_t (&acc)[C::TM][C::TN], uint4 *const (&xs)[4],
                                              uint4 *const (&ws)[4], const LoraEpilogue &ep,
                                              const RowTable<C> &rows, int M, int N, int n0, int tid,
                                              int lane, int wm0, int wn0) {
    lds_barrier();
    if (add_lora_steps<C, false, EXACT>(acc, xs, ws, ep, rows, M, N, n0, tid, lane, wm0, wn0))
        add_lora_steps<C, true, EXACT>(acc, xs, ws, ep, rows, M, N, n0, tid, lane, wm0, wn0);
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
