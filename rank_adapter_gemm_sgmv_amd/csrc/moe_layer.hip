// moe_layer.hip -- the two reductions of a whole mixture-of-experts layer (lora_moe_layer), each behind
// one launch of the expert-routed GEMM of moe.hip:
//
//   h[p] = act(g) * u,  g, u = the gate's and up's split sums + scale_i t B[i][e]     (pair p = (m, j))
//   y[m] = residual[m] + sum_j topk_w[m][j] (the down projection's split sums + scale_i t B[i][e])
//
// with t the adapter tiles' sums.  Everything is added in a fixed order: results do not depend on
// scheduling.  Both are bound by the length of their chain of dependent loads (routing and ids, then
// the adapter's rank and B), so a block loads the partial sums while it follows it.
#include "epilogue.h"

namespace lora {

namespace {

constexpr int kThreadsMoe = 256;

// One pair's adapter: its first rank row of B's pool (times the expert), rank and scale; rank 0 without.
struct PairAdapter {
    size_t row0;
    int rank;
    float scale;
};
__device__ __forceinline__ PairAdapter pair_adapter(const MoeLayerArgs &a, int e, int i) {
    PairAdapter p{0, 0, 0.0f};
    if (i >= 0 && i < a.n_adapters) {
        p.row0 = ((size_t)i * a.E + e) * a.r_stride;
        p.rank = a.ranks ? min(max(a.ranks[i], 0), a.r_stride) : a.r_stride;
        p.scale = a.scale[i];
    }
    return p;
}

// t[j] of pair p into LDS, by RM threads from `first` on
template <int RM>
__device__ __forceinline__ void pair_t(float *s_t, const MoeSums &s, int P, int p, int ks, int j) {
    if (j < 0 || j >= RM) return;
    float t = 0.0f;
    for (int sp = 0; sp < ks; ++sp) t += s.tpart[((size_t)sp * P + p) * RM + j];
    s_t[j] = t;
}

// z[4] = the splits of columns n .. n + 3 in order
__device__ __forceinline__ float4 split_sum(const MoeSums &s, int P, int p, int np, int ks, int n) {
    const float *q = s.partial + (size_t)p * np + n;
    float4 z = *reinterpret_cast<const float4 *>(q);
#pragma unroll 4
    for (int sp = 1; sp < ks; ++sp) {
        const float4 v = *reinterpret_cast<const float4 *>(q + (size_t)sp * P * np);
        z.x += v.x; z.y += v.y; z.z += v.z; z.w += v.w;
    }
    return z;
}

// z += scale t B[rows][n .. n + 3]
__device__ __forceinline__ void add_delta(float4 &z, const float *s_t, const uint16_t *B, const PairAdapter &ad,
                                          int N, int n) {
    const uint16_t *bp = B + ad.row0 * N + n;
    float4 d = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int j = 0; j < ad.rank; ++j) {
        const uint2 b = *reinterpret_cast<const uint2 *>(bp + (size_t)j * N);
        const float t = s_t[j];
        d.x = fmaf(t, bf16_lo(b.x), d.x); d.y = fmaf(t, bf16_hi(b.x), d.y);
        d.z = fmaf(t, bf16_lo(b.y), d.z); d.w = fmaf(t, bf16_hi(b.y), d.w);
    }
    z.x = fmaf(ad.scale, d.x, z.x); z.y = fmaf(ad.scale, d.y, z.y);
    z.z = fmaf(ad.scale, d.z, z.z); z.w = fmaf(ad.scale, d.w, z.w);
}

// Block (column chunk, pair), four columns per thread.
template <int RM, bool PARTS>
__global__ __launch_bounds__(kThreadsMoe) void moe_hidden_kernel(MoeLayerArgs a, MoeSums gate, MoeSums up, int N,
                                                                 int np, int ks, int act, uint16_t *h) {
    __shared__ float s_t[2][RM];
    const int p = blockIdx.y, e = a.topk_ids[p];
    if (e < 0 || e >= a.E) return;  // uniform in the block
    const int n = (blockIdx.x * kThreadsMoe + threadIdx.x) * 4;
    const bool ok = n < N;
    const int nc = ok ? n : 0;
    const PairAdapter ad = pair_adapter(a, e, a.ids[p / a.top_k]);
    float4 zg = split_sum(gate, a.P, p, np, ks, nc), zu = split_sum(up, a.P, p, np, ks, nc);
    if (ad.rank > 0) {  // uniform in the block
        pair_t<RM>(s_t[0], gate, a.P, p, ks, threadIdx.x);
        pair_t<RM>(s_t[1], up, a.P, p, ks, (int)threadIdx.x - 64);
        __syncthreads();
        add_delta(zg, s_t[0], gate.B, ad, N, nc);
        add_delta(zu, s_t[1], up.B, ad, N, nc);
    }
    if (!ok) return;
    float z[4] = {zg.x, zg.y, zg.z, zg.w};
    epi_act<4>(z, act);
    z[0] *= zu.x; z[1] *= zu.y; z[2] *= zu.z; z[3] *= zu.w;
    if constexpr (!PARTS) {
        // bf16: what the matrix instructions take; y's own rounding is as large
        *reinterpret_cast<uint2 *>(h + (size_t)p * N + n) = make_uint2(cvt_bf16x2(z[0], z[1]), cvt_bf16x2(z[2], z[3]));
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t b[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                b[v] = q < 3 ? bf16_part(z[v]) : 0u;
                z[v] = bf16_rest(z[v]);
            }
            *reinterpret_cast<uint2 *>(h + ((size_t)4 * p + q) * N + n) = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
        }
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
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = wave; j < a.top_k; j += NW) {
        const int p = m * a.top_k + j, e = a.topk_ids[p];
        if (e < 0 || e >= a.E) continue;  // uniform in the wave
        const PairAdapter ad = pair_adapter(a, e, i);
        float4 z = split_sum(down, a.P, p, np, ks, nc);
        if (ad.rank > 0) {
            // (LDS accesses of one wave complete in order; the compiler keeps them)
            pair_t<RM>(s_t[wave], down, a.P, p, ks, lane);
            __builtin_amdgcn_wave_barrier();
            add_delta(z, s_t[wave], down.B, ad, N, nc);
            __builtin_amdgcn_wave_barrier();
        }
        const float w = a.topk_w ? a.topk_w[p] : 1.0f;
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
    const size_t at = (size_t)m * N + n;
    if constexpr (YF32) {
        if (residual) {
            const float4 r = *reinterpret_cast<const float4 *>(static_cast<const float *>(residual) + at);
            sum.x += r.x; sum.y += r.y; sum.z += r.z; sum.w += r.w;
        }
        *reinterpret_cast<float4 *>(static_cast<float *>(y) + at) = sum;
    } else {
        if (residual) {
            const uint2 r = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(residual) + at);
            sum.x += bf16_lo(r.x); sum.y += bf16_hi(r.x); sum.z += bf16_lo(r.y); sum.w += bf16_hi(r.y);
        }
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(y) + at) =
            make_uint2(cvt_bf16x2(sum.x, sum.y), cvt_bf16x2(sum.z, sum.w));
    }
}

bool moe_args_ok(const MoePlan &p, const MoeLayerArgs &a, int N) {
    return a.P >= 1 && a.P <= LORA_MOE_MAX_PAIRS && N >= 4 && N % 4 == 0 && a.r_stride <= p.rm && p.ks >= 1;
}

}  // namespace

hipError_t launch_moe_hidden(const MoePlan &p, const MoeLayerArgs &a, const MoeSums &gate, const MoeSums &up,
                             int N, int act, bool parts, uint16_t *h, hipStream_t s) {
    if (!moe_args_ok(p, a, N)) return hipErrorInvalidValue;
    const dim3 grid((unsigned)((N + 4 * kThreadsMoe - 1) / (4 * kThreadsMoe)), (unsigned)a.P);
#define MOE_HIDDEN(RMX)                                                                          \
    if (parts) launch(moe_hidden_kernel<RMX, true>, grid, dim3(kThreadsMoe), 0, s, a, gate, up, N, p.np, p.ks, act, h); \
    else launch(moe_hidden_kernel<RMX, false>, grid, dim3(kThreadsMoe), 0, s, a, gate, up, N, p.np, p.ks, act, h)
    switch (p.rm) {
        case 8: MOE_HIDDEN(8); break;
        case 16: MOE_HIDDEN(16); break;
        case 32: MOE_HIDDEN(32); break;
        default: MOE_HIDDEN(64); break;
    }
#undef MOE_HIDDEN
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
