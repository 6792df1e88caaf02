// abi_driver.cpp -- the host side of liblora_mi355x (include/lora.h) under AddressSanitizer
// and UndefinedBehaviorSanitizer: every entry point called with arguments its validation
// rejects (and M = 0 no-ops), the sizing functions over many shapes, every status string.
// No call here reaches a kernel launch, so no GPU is needed; fake device addresses are never
// dereferenced.  Built by tests/test_sanitizers.py with the library's sources; exit status 0
// when every call returned the status expected of it.  Test infrastructure.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "lora.h"

static int failures = 0;
#define EXPECT(call, want)                                                                  \
    do {                                                                                    \
        int got_ = (int)(call);                                                             \
        if (got_ != (int)(want)) {                                                          \
            fprintf(stderr, "%s:%d: %s returned %d, expected %d\n", __FILE__, __LINE__, #call, \
                    got_, (int)(want));                                                     \
            ++failures;                                                                     \
        }                                                                                   \
    } while (0)

static void *const F = reinterpret_cast<void *>(uintptr_t(1) << 20);  // 256-byte aligned
static float *const FF = static_cast<float *>(F);
static int32_t *const FI = static_cast<int32_t *>(F);
static void *off(size_t b) { return static_cast<char *>(F) + b; }

int main() {
    // sizing
    EXPECT(lora_max_tiles(0, 4), 0);
    EXPECT(lora_max_tiles(16, 4), 5);
    EXPECT(lora_max_tiles(-3, 4), 0);
    const int rs[] = {0, 1, 7, 8, 12, 16, 24, 33, 64, 65};
    const int Ms[] = {0, 1, 64, 128, 129, 256, 257, 767, 768, 1024, 4096};
    const int ds[] = {8, 120, 4096, 4104, 11008};
    for (int r : rs)
        for (int M : Ms)
            for (int d : ds) {
                const size_t b = lora_workspace_bytes(M, d, 4096, r, 32);
                const bool ok = r >= 1 && r <= 64;
                if ((b != 0) != (ok && M > 0) || b % 256 != 0) {
                    fprintf(stderr, "workspace bytes %zu for M %d d %d r %d\n", b, M, d, r);
                    ++failures;
                }
            }
    for (int r : rs)
        for (int M : {0, 1, 64, 2048, 2049})
            for (int E : {0, 1, 32, 4096, 4097}) {
                const size_t b = lora_moe_workspace_bytes(M, 4, E, 2880, 2880, r, 8);
                const bool ok = r >= 8 && r % 8 == 0 && r <= 64 && M > 0 && M <= 2048 && E >= 1 &&
                                E <= 4096;
                if ((b != 0) != ok || b % 256 != 0) {
                    fprintf(stderr, "moe workspace bytes %zu for M %d E %d r %d\n", b, M, E, r);
                    ++failures;
                }
            }
    for (int s = -1; s <= 12; ++s) {
        const char *str = lora_status_string(static_cast<lora_status_t>(s));
        if (!str || !*str) ++failures;
    }
    if (!lora_last_hip_error()) ++failures;

    lora_segments_t seg{FI, FI, FI, FI, FI};
    lora_segments_t bad_seg{FI, nullptr, FI, FI, FI};
    const size_t ws = lora_workspace_bytes(64, 4096, 4096, 16, 32);

    // segments
    EXPECT(lora_build_segments(FI, -1, 8, seg, nullptr), LORA_ERR_SHAPE);
    EXPECT(lora_build_segments(FI, 8, 0, seg, nullptr), LORA_ERR_SHAPE);
    EXPECT(lora_build_segments(nullptr, 8, 4, seg, nullptr), LORA_ERR_NULL);
    EXPECT(lora_build_segments(FI, 8, 4, bad_seg, nullptr), LORA_ERR_NULL);
    EXPECT(lora_build_segments(static_cast<int32_t *>(off(2)), 8, 4, seg, nullptr), LORA_ERR_ALIGN);
    EXPECT(lora_build_segments(FI, 0, 4, seg, nullptr), LORA_OK);

    // shrink / expand (padded and compact)
    EXPECT(lora_shrink(F, F, nullptr, 64, 4096, 65, 32, seg, FF, F, ws, nullptr), LORA_ERR_RANK);
    EXPECT(lora_shrink(F, F, nullptr, 64, 12, 16, 32, seg, FF, F, ws, nullptr), LORA_ERR_SHAPE);
    EXPECT(lora_shrink(nullptr, F, nullptr, 64, 4096, 16, 32, seg, FF, F, ws, nullptr), LORA_ERR_NULL);
    EXPECT(lora_shrink(F, F, nullptr, 64, 4096, 16, 32, seg, FF, F, 16, nullptr), LORA_ERR_WORKSPACE);
    EXPECT(lora_shrink_compact(F, F, FI, nullptr, 64, 64, 4096, 16, 32, seg, FF, F, ws, nullptr),
           LORA_ERR_NULL);
    EXPECT(lora_shrink_compact(F, F, FI, FI, 0, 64, 4096, 16, 32, seg, FF, F, ws, nullptr),
           LORA_ERR_SHAPE);
    EXPECT(lora_expand(FF, F, FF, nullptr, 64, 4096, 16, 32, seg, F, static_cast<lora_dtype_t>(3),
                       nullptr), LORA_ERR_DTYPE);
    EXPECT(lora_expand(FF, F, FF, nullptr, 64, 4100, 16, 32, seg, F, LORA_BF16, nullptr),
           LORA_ERR_SHAPE);
    EXPECT(lora_expand_compact(FF, F, FF, FI, FI, 1 << 20, 64, 4096, 16, 32, seg, F, LORA_BF16,
                               nullptr), LORA_ERR_SHAPE);

    // the layer and its variants
    const lora_mode_t dec = LORA_MODE_DECODE;
    EXPECT(lora_linear(F, F, F, F, FF, nullptr, FI, -1, 4096, 4096, 16, 32, nullptr, F, LORA_BF16,
                       dec, F, ws, nullptr), LORA_ERR_SHAPE);
    EXPECT(lora_linear(F, F, F, F, FF, nullptr, FI, 64, 4096, 4096, 0, 32, nullptr, F, LORA_BF16,
                       dec, F, ws, nullptr), LORA_ERR_RANK);
    EXPECT(lora_linear(F, F, F, F, FF, nullptr, FI, 64, 4096, 4096, 16, 32, nullptr, F, LORA_BF16,
                       static_cast<lora_mode_t>(7), F, ws, nullptr), LORA_ERR_MODE);
    EXPECT(lora_linear(F, F, F, F, FF, nullptr, nullptr, 64, 4096, 4096, 16, 32, nullptr, F,
                       LORA_BF16, dec, F, ws, nullptr), LORA_ERR_NULL);
    EXPECT(lora_linear(off(2), F, F, F, FF, nullptr, FI, 64, 4096, 4096, 16, 32, nullptr, F,
                       LORA_BF16, dec, F, ws, nullptr), LORA_ERR_ALIGN);
    EXPECT(lora_linear(F, F, F, F, FF, nullptr, FI, 64, 4096, 4096, 16, 32, &bad_seg, F, LORA_BF16,
                       dec, F, ws, nullptr), LORA_ERR_NULL);
    EXPECT(lora_linear(F, F, F, F, FF, nullptr, FI, 64, 4096, 4096, 16, 32, nullptr, F, LORA_BF16,
                       dec, F, ws - 1, nullptr), LORA_ERR_WORKSPACE);
    EXPECT(lora_linear(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, 4096, 4096,
                       16, 32, nullptr, nullptr, LORA_BF16, dec, nullptr, 0, nullptr), LORA_OK);
    EXPECT(lora_linear_compact(F, F, F, F, FF, FI, FI, 0, FI, 64, 4096, 4096, 16, 32, nullptr, F,
                               LORA_BF16, dec, F, ws, nullptr), LORA_ERR_SHAPE);
    EXPECT(lora_linear_compact(F, F, F, F, FF, nullptr, FI, 64, FI, 64, 4096, 4096, 16, 32, nullptr,
                               F, LORA_BF16, dec, F, ws, nullptr), LORA_ERR_NULL);
    EXPECT(lora_linear_noalloc(F, F, F, F, FF, nullptr, FI, 512, 4096, 11008, 16, 32, nullptr, F,
                               LORA_BF16, dec, nullptr), LORA_ERR_WORKSPACE);
    EXPECT(lora_linear_noalloc(F, F, F, F, FF, nullptr, FI, 64, 4096, 4096, 99, 32, nullptr, F,
                               LORA_BF16, dec, nullptr), LORA_ERR_RANK);
    EXPECT(lora_linear_fp8w(F, F, FF, F, F, FF, nullptr, FI, 257, 4096, 4096, 16, 32, nullptr, F,
                            LORA_BF16, dec, F, ws, nullptr), LORA_ERR_SHAPE);
    EXPECT(lora_linear_fp8w(F, F, FF, F, F, FF, nullptr, FI, 64, 4096, 4096, 16, 32, nullptr, F,
                            LORA_BF16, LORA_MODE_PREFILL, F, ws, nullptr), LORA_ERR_MODE);
    EXPECT(lora_linear_fp8w(F, F, nullptr, F, F, FF, nullptr, FI, 64, 4096, 4096, 16, 32, nullptr,
                            F, LORA_BF16, dec, F, ws, nullptr), LORA_ERR_NULL);

    // measurement aids: their own argument checks first, then the call's validation
    float ms[4];
    const char *names[4];
    int32_t nk = 7;
    EXPECT(lora_linear_profiled(F, F, F, F, FF, nullptr, FI, 64, 4096, 4096, 16, 32, nullptr, F,
                                LORA_BF16, dec, F, ws, nullptr, nullptr, names, 4, &nk),
           LORA_ERR_NULL);
    EXPECT(lora_linear_profiled(F, F, F, F, FF, nullptr, FI, 64, 4096, 4096, 16, 32, nullptr, F,
                                LORA_BF16, dec, F, 8, nullptr, ms, names, 4, &nk),
           LORA_ERR_WORKSPACE);
    EXPECT(nk, 0);
    EXPECT(lora_linear_compact_profiled(F, F, F, F, FF, FI, FI, 0, FI, 64, 4096, 4096, 16, 32,
                                        nullptr, F, LORA_BF16, dec, F, ws, nullptr, ms, names, 4,
                                        &nk), LORA_ERR_SHAPE);
    EXPECT(lora_linear_fp8w_profiled(F, F, FF, F, F, FF, nullptr, FI, 64, 4100, 4096, 16, 32,
                                     nullptr, F, LORA_BF16, dec, F, ws, nullptr, ms, names, 4, &nk),
           LORA_ERR_SHAPE);

    // MoE
    const size_t mws = lora_moe_workspace_bytes(64, 4, 32, 2880, 2880, 16, 8);
    EXPECT(lora_moe_linear(F, F, F, F, FF, nullptr, FI, FI, FF, 64, 4, 32, 2880, 2880, 12, 8, F,
                           LORA_BF16, dec, F, mws, nullptr), LORA_ERR_RANK);
    EXPECT(lora_moe_linear(F, F, F, F, FF, nullptr, FI, FI, FF, 2049, 4, 32, 2880, 2880, 16, 8, F,
                           LORA_BF16, dec, F, mws, nullptr), LORA_ERR_SHAPE);
    EXPECT(lora_moe_linear(F, F, F, F, FF, nullptr, FI, nullptr, FF, 64, 4, 32, 2880, 2880, 16, 8,
                           F, LORA_BF16, dec, F, mws, nullptr), LORA_ERR_NULL);
    EXPECT(lora_moe_linear(F, F, F, F, FF, nullptr, FI, FI, static_cast<float *>(off(2)), 64, 4, 32,
                           2880, 2880, 16, 8, F, LORA_BF16, dec, F, mws, nullptr), LORA_ERR_ALIGN);
    EXPECT(lora_moe_linear(F, F, F, F, FF, nullptr, FI, FI, FF, 64, 4, 32, 2880, 2880, 16, 8, F,
                           LORA_BF16, dec, F, mws - 1, nullptr), LORA_ERR_WORKSPACE);
    EXPECT(lora_moe_linear(F, F, F, F, FF, nullptr, FI, FI, FF, 64, 4, 32, 2880, 2880, 16, 8, F,
                           LORA_BF16, LORA_MODE_PREFILL, F, mws, nullptr), LORA_ERR_MODE);
    EXPECT(lora_moe_linear(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                           nullptr, 0, 4, 32, 2880, 2880, 16, 8, nullptr, LORA_BF16, dec, nullptr,
                           0, nullptr), LORA_OK);
    EXPECT(lora_moe_linear_profiled(F, F, F, F, FF, nullptr, FI, FI, FF, 64, 4, 32, 2880, 2880, 16,
                                    8, F, LORA_BF16, dec, F, mws, nullptr, ms, names, -1, &nk),
           LORA_ERR_NULL);

    // several projections
    {
        const void *const in[2] = {F, F};
        void *const out[2] = {F, F}, *const bad_out[2] = {F, off(8)};
        for (int np : {-1, 0, 1, 2, LORA_MAX_PROJ, LORA_MAX_PROJ + 1})
            for (int r : rs)
                for (int M : {0, 1, 200, 512, 4096, LORA_MAX_ROWS, LORA_MAX_ROWS + 1})
                    for (int d : {8, 12, 4096, 4104, 1 << 20}) {
                        const size_t b = lora_workspace_bytes_multi(M, d, 4096, r, 32, np);
                        const bool ok = np >= 1 && np <= LORA_MAX_PROJ && r >= 1 && r <= 64 && M > 0 &&
                                        M <= LORA_MAX_ROWS && d % 8 == 0;
                        if ((b != 0) != ok || b % 256 != 0) {
                            fprintf(stderr, "multi workspace bytes %zu for M %d d %d r %d n %d\n", b, M, d, r, np);
                            ++failures;
                        }
                    }
        const size_t w2 = lora_workspace_bytes_multi(512, 4096, 4096, 16, 32, 2);
        EXPECT(lora_linear_multi(F, 0, in, in, in, FF, nullptr, FI, 512, 4096, 4096, 16, 32, nullptr, out,
                                 LORA_BF16, dec, F, w2, nullptr), LORA_ERR_SHAPE);
        EXPECT(lora_linear_multi(F, 2, nullptr, in, in, FF, nullptr, FI, 512, 4096, 4096, 16, 32, nullptr,
                                 out, LORA_BF16, dec, F, w2, nullptr), LORA_ERR_NULL);
        EXPECT(lora_linear_multi(F, 2, in, in, in, FF, nullptr, FI, 512, 4096, 4096, 16, 32, nullptr, bad_out,
                                 LORA_BF16, dec, F, w2, nullptr), LORA_ERR_ALIGN);
        EXPECT(lora_linear_multi(F, 2, in, in, in, FF, nullptr, FI, 512, 4096, 4096, 16, 32, nullptr, out,
                                 LORA_BF16, dec, F, w2 - 1, nullptr), LORA_ERR_WORKSPACE);
        EXPECT(lora_linear_multi_profiled(F, 2, in, in, in, FF, nullptr, FI, 512, 4096, 4096, 16, 32, nullptr,
                                          out, LORA_BF16, dec, F, w2 - 1, nullptr, ms, names, 4, &nk),
               LORA_ERR_WORKSPACE);
        EXPECT(lora_linear_multi(nullptr, 2, in, in, in, nullptr, nullptr, nullptr, 0, 4096, 4096, 16, 32,
                                 nullptr, out, LORA_BF16, dec, nullptr, 0, nullptr), LORA_OK);
    }

    // the layer with an epilogue
    const auto act = [&](const lora_epilogue_t *e, int M, int d, const void *x, void *y, size_t nb) {
        return lora_linear_act(x, F, F, F, FF, nullptr, FI, M, d, 4096, 16, 32, nullptr, e, y, LORA_BF16, dec, F,
                               nb, nullptr);
    };
    EXPECT(act(nullptr, -1, 4096, F, F, ws), LORA_ERR_SHAPE);
    EXPECT(act(nullptr, LORA_MAX_ROWS + 1, 4096, F, F, ws), LORA_ERR_SHAPE);
    EXPECT(act(nullptr, 64, 12, F, F, ws), LORA_ERR_SHAPE);
    EXPECT(act(nullptr, 64, 4096, nullptr, F, ws), LORA_ERR_NULL);
    EXPECT(act(nullptr, 64, 4096, F, nullptr, ws), LORA_ERR_NULL);
    EXPECT(act(nullptr, 64, 4096, F, off(8), ws), LORA_ERR_ALIGN);
    EXPECT(act(nullptr, 64, 4096, F, F, ws - 1), LORA_ERR_WORKSPACE);
    for (int M : {64, 0}) {
        for (int a : {-1, 5, 1 << 30}) {
            const lora_epilogue_t e{nullptr, nullptr, nullptr, static_cast<lora_act_t>(a)};
            EXPECT(act(&e, M, 4096, F, F, ws), LORA_ERR_VALUE);
        }
        for (int k = 0; k < 3; ++k) {
            const void *p[3] = {F, nullptr, F};
            p[k] = off(8);
            const lora_epilogue_t e{p[0], p[1], p[2], LORA_ACT_SILU};
            EXPECT(act(&e, M, 4096, F, F, ws), LORA_ERR_ALIGN);
        }
        const lora_epilogue_t e{F, F, F, LORA_ACT_GELU};
        EXPECT(act(&e, M, 4096, nullptr, F, ws), M ? LORA_ERR_NULL : LORA_OK);
    }

    // the layer on 8-bit operands
    for (int r : rs)
        for (int M : {-1, 0, 1, 64, 128, 129, 192, 193, 256, 257, 1024, 4096, LORA_MAX_ROWS, LORA_MAX_ROWS + 1})
            for (int d : {-16, 0, 8, 16, 120, 128, 136, 4096, 4104, 11008, 1 << 20, (1 << 20) + 16})
                for (int n : {8, 12, 4104, 1 << 20})
                    for (int na : {0, 1, 256, LORA_MAX_ADAPTERS}) {
                        const size_t b = lora_fp8_workspace_bytes(M, d, n, r, na);
                        const bool ok = r >= 1 && r <= 64 && M > 0 && M <= LORA_MAX_ROWS && d > 0 && d % 16 == 0 &&
                                        d <= 1 << 20 && n % 8 == 0 && na >= 1;
                        if ((b != 0) != ok || b % 256 != 0) {
                            fprintf(stderr, "fp8 workspace bytes %zu for M %d d %d x %d r %d n %d\n", b, M, d, n, r, na);
                            ++failures;
                        }
                    }
    const size_t fws = lora_fp8_workspace_bytes(64, 4096, 4096, 16, 32);
    const auto fp8 = [&](const lora_epilogue_t *e, int M, int d, const void *x8, const float *xs, lora_mode_t mode,
                         size_t nb) {
        return lora_linear_fp8(x8, xs, F, FF, F, F, FF, nullptr, FI, M, d, 4096, 16, 32, nullptr, e, F, LORA_BF16,
                               mode, F, nb, nullptr);
    };
    const lora_mode_t any = LORA_MODE_AUTO;
    EXPECT(fp8(nullptr, 64, 4104, F, FF, any, fws), LORA_ERR_SHAPE);
    EXPECT(fp8(nullptr, LORA_MAX_ROWS + 1, 4096, F, FF, any, fws), LORA_ERR_SHAPE);
    EXPECT(fp8(nullptr, 64, 4096, F, FF, dec, fws), LORA_ERR_MODE);
    EXPECT(fp8(nullptr, 64, 4096, F, FF, static_cast<lora_mode_t>(LORA_MODE_PREFILL | LORA_MODE_CHECKED), fws),
           LORA_ERR_MODE);
    EXPECT(fp8(nullptr, 64, 4096, nullptr, FF, any, fws), LORA_ERR_NULL);
    EXPECT(fp8(nullptr, 64, 4096, F, nullptr, any, fws), LORA_ERR_NULL);
    EXPECT(fp8(nullptr, 64, 4096, off(8), FF, any, fws), LORA_ERR_ALIGN);
    EXPECT(fp8(nullptr, 64, 4096, F, static_cast<float *>(off(2)), any, fws), LORA_ERR_ALIGN);
    EXPECT(fp8(nullptr, 64, 4096, F, FF, any, fws - 1), LORA_ERR_WORKSPACE);
    {
        const lora_epilogue_t bad_act{nullptr, nullptr, nullptr, static_cast<lora_act_t>(9)};
        const lora_epilogue_t bad_mul{nullptr, off(4), nullptr, LORA_ACT_NONE};
        EXPECT(fp8(&bad_act, 64, 4096, F, FF, any, fws), LORA_ERR_VALUE);
        EXPECT(fp8(&bad_mul, 0, 4096, F, FF, any, fws), LORA_ERR_ALIGN);
        EXPECT(fp8(nullptr, 0, 4096, nullptr, nullptr, any, 0), LORA_OK);
    }

    // the norm in front of it
    const auto norm = [&](const void *x, float eps, int M, int d, void *y, void *y8, float *ys) {
        return lora_rmsnorm(x, F, F, eps, M, d, F, y, y8, ys, nullptr);
    };
    EXPECT(norm(F, 1e-5f, -1, 64, F, F, FF), LORA_ERR_SHAPE);
    EXPECT(norm(F, 1e-5f, LORA_MAX_ROWS + 1, 64, F, F, FF), LORA_ERR_SHAPE);
    EXPECT(norm(F, 1e-5f, 4, 60, F, F, FF), LORA_ERR_SHAPE);
    EXPECT(norm(F, 1e-5f, 4, (1 << 20) + 8, F, F, FF), LORA_ERR_SHAPE);
    EXPECT(norm(F, 0.0f, 4, 64, F, F, FF), LORA_ERR_VALUE);
    EXPECT(norm(F, __builtin_nanf(""), 4, 64, F, F, FF), LORA_ERR_VALUE);
    EXPECT(norm(F, __builtin_inff(), 4, 64, F, F, FF), LORA_ERR_VALUE);
    EXPECT(norm(nullptr, 1e-5f, 4, 64, F, F, FF), LORA_ERR_NULL);
    EXPECT(norm(F, 1e-5f, 4, 64, nullptr, nullptr, nullptr), LORA_ERR_NULL);
    EXPECT(norm(F, 1e-5f, 4, 64, F, F, nullptr), LORA_ERR_NULL);
    EXPECT(norm(F, 1e-5f, 4, 64, F, nullptr, FF), LORA_ERR_NULL);
    EXPECT(norm(off(8), 1e-5f, 4, 64, F, F, FF), LORA_ERR_ALIGN);
    EXPECT(norm(F, 1e-5f, 4, 64, F, off(8), FF), LORA_ERR_ALIGN);
    EXPECT(norm(F, 1e-5f, 4, 64, F, F, static_cast<float *>(off(2))), LORA_ERR_ALIGN);
    EXPECT(norm(nullptr, 1e-5f, 0, 64, nullptr, nullptr, nullptr), LORA_OK);

    if (failures) {
        fprintf(stderr, "%d unexpected results\n", failures);
        return 1;
    }
    printf("abi driver: all calls returned the expected status\n");
    return 0;
}
