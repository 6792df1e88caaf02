// moe_layer.hip -- the two reductions of a whole mixture-of-experts layer (lora_moe_layer), each behind
// one launch of the expert-routed GEMM of moe.hip:
//
//   h[p] = act(g) * u,  g, u = the gate's and up's split sums + scale_i t B[i][e]     (pair p = (m, j))
//   y[m] = residual[m] + sum_j topk_w[m][j] (the down projection's split sums + scale_i t B[i][e])
//
// with t the adapter tiles' sums.  Everything is added in a fixed order: results do not depend on
// scheduling.  Both are bound by the length of their chain of dependent loads (routing and ids, then
// the adapter's rank and B), so a block loads the partial sums while it follows it.  us of hidden and out: one
// token, 4 of 32 experts of 2880 x 2880 4.7 and 4.6; 64 tokens 9.5 and 6.7; 23 tokens, 2 of 8 experts of 1040 x
// 2768, fp32 6.4 and 5.2.
#include "epilogue.h"

namespace lora {

namespace {

constexpr int kThreadsMoe = 256;

// Four columns of one pair: the splits in order, plus scale_i t B[i][e].  Called by a group of at least
// RM threads (thread `tj` of it) that share s_t and meet at sync(); every load whose address is known
// is issued before the first wait: the partial sums, t's parts and the first eight rows of B together
// (rows past the adapter's rank are not used); B's other rows, as many as the rank has, once that is
// here.  Many pairs read many different B: all rows of the stride at once took 304 us in
// 64 tokens' layer of 32 experts of 2880 x 2880 (8 adapters of ranks 1-16) where the ranks' own take 302.
template <int RM, class F>
__device__ __forceinline__ float4 pair_columns(const MoeLayerArgs &a, const MoeSums &s, int p, int e, int i, int np,
                                               int ks, int N, int n, float *s_t, int tj, F sync) {
    constexpr int FIRST = 8, REST = RM - FIRST, EARLY = 4;
    const float *q = s.partial + (size_t)p * np + n;
    const size_t qs = (size_t)a.P * np, ts = (size_t)a.P * RM;
    float4 pv[EARLY];
#pragma unroll
    for (int sp = 0; sp < EARLY; ++sp)
        if (sp < ks) pv[sp] = *reinterpret_cast<const float4 *>(q + sp * qs);
    const bool has = i >= 0 && i < a.n_adapters;  // uniform in the group
    const int ad = has ? i : 0;
    int rank = 0;
    float scale = 0.0f;
    const uint16_t *bp = s.B + ((size_t)ad * a.E + e) * a.r_stride * N + n;
    uint2 bv[FIRST], br[REST > 0 ? REST : 1];
    if (has) {
        rank = a.ranks ? min(max(a.ranks[ad], 0), a.r_stride) : a.r_stride;
        scale = a.scale[ad];
#pragma unroll
        for (int j = 0; j < FIRST; ++j) bv[j] = *reinterpret_cast<const uint2 *>(bp + (size_t)j * N);
        if (tj < RM) {
            const float *tp = s.tpart + (size_t)p * RM + tj;
            float tv[EARLY], t = 0.0f;
#pragma unroll
            for (int sp = 0; sp < EARLY; ++sp) tv[sp] = sp < ks ? tp[sp * ts] : 0.0f;
#pragma unroll
            for (int sp = 0; sp < EARLY; ++sp)
                if (sp < ks) t += tv[sp];
            for (int sp = EARLY; sp < ks; ++sp) t += tp[sp * ts];
            s_t[tj] = t;
        }
#pragma unroll
        for (int j = 0; j < REST; ++j)
            if (FIRST + j < rank) br[j] = *reinterpret_cast<const uint2 *>(bp + (size_t)(FIRST + j) * N);
    }
    sync();
    float4 z = pv[0];
#pragma unroll
    for (int sp = 1; sp < EARLY; ++sp)
        if (sp < ks) { z.x += pv[sp].x; z.y += pv[sp].y; z.z += pv[sp].z; z.w += pv[sp].w; }
    for (int sp = EARLY; sp < ks; ++sp) {
        const float4 v = *reinterpret_cast<const float4 *>(q + sp * qs);
        z.x += v.x; z.y += v.y; z.z += v.z; z.w += v.w;
    }
    if (has) {
        float4 d = make_float4(0.f, 0.f, 0.f, 0.f);
        auto row = [&](int j, uint2 b) {
            const float t = s_t[j];
            d.x = fmaf(t, bf16_lo(b.x), d.x); d.y = fmaf(t, bf16_hi(b.x), d.y);
            d.z = fmaf(t, bf16_lo(b.y), d.z); d.w = fmaf(t, bf16_hi(b.y), d.w);
        };
        // (the rank is uniform in the group)
#pragma unroll
        for (int j = 0; j < FIRST; ++j)
            if (j < rank) row(j, bv[j]);
#pragma unroll
        for (int j = 0; j < REST; ++j)
            if (FIRST + j < rank) row(FIRST + j, br[j]);
        z.x = fmaf(scale, d.x, z.x); z.y = fmaf(scale, d.y, z.y);
        z.z = fmaf(scale, d.z, z.z); z.w = fmaf(scale, d.w, z.w);
    }
    return z;
}

// Block (chunk of 512 columns, pair), four columns per thread: the first half of the block sums the
// gate, the second up, which it hands over through LDS.
template <int RM, MoeRows ROWS>
__global__ __launch_bounds__(kThreadsMoe) void moe_hidden_kernel(MoeLayerArgs a, MoeSums gate, MoeSums up, int N,
                                                                 int np, int ks, int act, uint16_t *h) {
    constexpr int HALF = kThreadsMoe / 2;
    static_assert(HALF >= 64, "RM threads of each half sum t");
    __shared__ float s_t[2][RM];
    __shared__ float4 s_up[HALF];
    const int p = blockIdx.y, e = a.topk_ids[p], i = a.ids[p / a.top_k];
    if (e < 0 || e >= a.E) return;  // uniform in the block
    const int which = threadIdx.x / HALF, t = threadIdx.x % HALF;  // (uniform in a wave)
    const int n = (blockIdx.x * HALF + t) * 4;
    const bool ok = n < N;
    const float4 v = pair_columns<RM>(a, which ? up : gate, p, e, i, np, ks, N, ok ? n : 0, s_t[which], t,
                                      [] { __syncthreads(); });
    if (which) s_up[t] = v;
    __syncthreads();
    if (which || !ok) return;
    const float4 zu = s_up[t];
    float z[4] = {v.x, v.y, v.z, v.w};
    epi_act<4>(z, act);
    z[0] *= zu.x; z[1] *= zu.y; z[2] *= zu.z; z[3] *= zu.w;
    // The matrix instructions take bf16, a value's parts add up in fp32: two of them for y in bf16, whose own
    // rounding is 2^8 times as large as what they leave out; with y in fp32 nothing is.
    constexpr int NP = moe_rows_of_pair(ROWS);
#pragma unroll
    for (int q = 0; q < NP; ++q) {
        uint32_t b[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            b[c] = q < 3 ? bf16_part(z[c]) : 0u;
            z[c] = bf16_rest(z[c]);
        }
        *reinterpret_cast<uint2 *>(h + ((size_t)NP * p + q) * N + n) =
            make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
    }
}

// Block (chunk of 256 columns, token): wave w takes the token's slots w, w + 4, ..., four columns per
// lane; the waves' sums are added in wave order.
template <int RM, bool YF32>
__global__ __launch_bounds__(kThreadsMoe) void moe_out_kernel(MoeLayerArgs a, MoeSums down, int N, int np, int ks,
                                                              const void *residual, void *y) {
    constexpr int NW = kThreadsMoe / 64;
    __shared__ float s_t[NW][RM];
    __shared__ float4 s_z[NW][64];
    const int m = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = (blockIdx.x * 64 + lane) * 4;
    const bool ok = n < N;
    const int nc = ok ? n : 0;
    const int i = a.ids[m];
    const size_t at = (size_t)m * N + n;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f), res = sum;
    if (residual && wave == 0 && ok) {
        if constexpr (YF32) {
            res = *reinterpret_cast<const float4 *>(static_cast<const float *>(residual) + at);
        } else {
            const uint2 r = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(residual) + at);
            res = make_float4(bf16_lo(r.x), bf16_hi(r.x), bf16_lo(r.y), bf16_hi(r.y));
        }
    }
    for (int j = wave; j < a.top_k; j += NW) {
        const int p = m * a.top_k + j, e = a.topk_ids[p];
        const float w = a.topk_w ? a.topk_w[p] : 1.0f;
        if (e < 0 || e >= a.E) continue;  // uniform in the wave
        // (a wave's LDS accesses complete in order)
        const float4 z = pair_columns<RM>(a, down, p, e, i, np, ks, N, nc, s_t[wave], lane,
                                          [] { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); __builtin_amdgcn_wave_barrier(); });
        __builtin_amdgcn_wave_barrier();
        sum.x = fmaf(w, z.x, sum.x); sum.y = fmaf(w, z.y, sum.y);
        sum.z = fmaf(w, z.z, sum.z); sum.w = fmaf(w, z.w, sum.w);
    }
    s_z[wave][lane] = sum;
    __syncthreads();
    if (wave != 0 || !ok) return;
#pragma unroll
    for (int w = 1; w < NW; ++w) {
        const float4 v = s_z[w][lane];
        sum.x += v.x; sum.y += v.y; sum.z += v.z; sum.w += v.w;
    }
    sum.x += res.x; sum.y += res.y; sum.z += res.z; sum.w += res.w;
    if constexpr (YF32)
        *reinterpret_cast<float4 *>(static_cast<float *>(y) + at) = sum;
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(y) + at) =
            make_uint2(cvt_bf16x2(sum.x, sum.y), cvt_bf16x2(sum.z, sum.w));
}

bool moe_args_ok(const MoePlan &p, const MoeLayerArgs &a, int N) {
    return a.P >= 1 && a.P <= LORA_MOE_MAX_PAIRS && N >= 4 && N % 4 == 0 && a.r_stride <= p.rm && p.ks >= 1;
}

}  // namespace

hipError_t launch_moe_hidden(const MoePlan &p, const MoeLayerArgs &a, const MoeSums &gate, const MoeSums &up,
                             int N, int act, MoeRows rows, uint16_t *h, hipStream_t s) {
    if (!moe_args_ok(p, a, N) || rows == kMoeToken) return hipErrorInvalidValue;
    const dim3 grid((unsigned)((N + 2 * kThreadsMoe - 1) / (2 * kThreadsMoe)), (unsigned)a.P);
#define MOE_HIDDEN_ONE(RMX, ROWS)                                                                \
    launch(moe_hidden_kernel<RMX, ROWS>, grid, dim3(kThreadsMoe), 0, s, a, gate, up, N, p.np, p.ks, act, h)
#define MOE_HIDDEN(RMX)                                                                          \
    if (rows == kMoeParts4) MOE_HIDDEN_ONE(RMX, kMoeParts4);                                     \
    else MOE_HIDDEN_ONE(RMX, kMoeParts2)
    switch (p.rm) {
        case 8: MOE_HIDDEN(8); break;
        case 16: MOE_HIDDEN(16); break;
        case 32: MOE_HIDDEN(32); break;
        default: MOE_HIDDEN(64); break;
    }
#undef MOE_HIDDEN
#undef MOE_HIDDEN_ONE
    return hipGetLastError();
}

hipError_t launch_moe_out(const MoePlan &p, const MoeLayerArgs &a, const MoeSums &down, int M, int N,
                          const void *residual, void *y, bool y_f32, hipStream_t s) {
    if (!moe_args_ok(p, a, N) || M < 1) return hipErrorInvalidValue;
    const dim3 grid((unsigned)((N + 255) / 256), (unsigned)M);
#define MOE_OUT(RMX)                                                                             \
    if (y_f32) launch(moe_out_kernel<RMX, true>, grid, dim3(kThreadsMoe), 0, s, a, down, N, p.np, p.ks, residual, y); \
    else launch(moe_out_kernel<RMX, false>, grid, dim3(kThreadsMoe), 0, s, a, down, N, p.np, p.ks, residual, y)
    switch (p.rm) {
        case 8: MOE_OUT(8); break;
        case 16: MOE_OUT(16); break;
        case 32: MOE_OUT(32); break;
        default: MOE_OUT(64); break;
    }
#undef MOE_OUT
    return hipGetLastError();
}

}  // namespace lora
