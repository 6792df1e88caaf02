// abi_more_driver.cpp -- the host side of the rows in 8-bit integers, the layer on them, the expert layer
// and the rotary positions (include/lora.h) under AddressSanitizer and UndefinedBehaviorSanitizer: what
// their validation rejects, M = 0 no-ops, and the sizing functions up to the limits.  No call here
// reaches a kernel launch; fake device addresses are never dereferenced.  Built by
// tests/test_sanitizers_more.py; exit status 0 when every call returned the status expected of it.
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

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

static void rows() {
    const auto norm = [&](const void *x, float eps, int M, int d, void *y8, float *ys) {
        return lora_rmsnorm_int8(x, F, F, eps, M, d, F, F, y8, ys, nullptr);
    };
    for (int M : {INT_MIN, -1, LORA_MAX_ROWS + 1, INT_MAX}) {
        EXPECT(norm(F, 1e-5f, M, 64, F, FF), LORA_ERR_SHAPE);
        EXPECT(lora_quant_int8(F, M, 64, F, FF, nullptr), LORA_ERR_SHAPE);
    }
    for (int d : {INT_MIN, -8, 0, 12, (1 << 20) + 8, INT_MAX}) {
        EXPECT(norm(F, 1e-5f, 4, d, F, FF), LORA_ERR_SHAPE);
        EXPECT(lora_quant_int8(F, 4, d, F, FF, nullptr), LORA_ERR_SHAPE);
    }
    EXPECT(norm(F, 0.0f, 4, 64, F, FF), LORA_ERR_VALUE);
    EXPECT(norm(F, NAN, 4, 64, F, FF), LORA_ERR_VALUE);
    EXPECT(norm(nullptr, 1e-5f, 4, 64, F, FF), LORA_ERR_NULL);
    EXPECT(norm(F, 1e-5f, 4, 64, nullptr, nullptr), LORA_ERR_NULL);
    EXPECT(norm(F, 1e-5f, 4, 64, F, nullptr), LORA_ERR_NULL);
    EXPECT(norm(F, 1e-5f, 4, 64, off(8), FF), LORA_ERR_ALIGN);
    EXPECT(lora_quant_int8(F, 4, 64, nullptr, FF, nullptr), LORA_ERR_NULL);
    EXPECT(lora_quant_int8(F, 4, 64, F, static_cast<float *>(off(2)), nullptr), LORA_ERR_ALIGN);
    EXPECT(lora_quant_int8(off(2), 4, 64, F, FF, nullptr), LORA_ERR_ALIGN);
    EXPECT(norm(nullptr, 1e-5f, 0, 64, nullptr, nullptr), LORA_OK);
    EXPECT(lora_quant_int8(nullptr, 0, 64, nullptr, nullptr, nullptr), LORA_OK);
}

static void layer() {
    for (int r : {INT_MIN, 0, 1, 8, 24, 64, 65, INT_MAX})
        for (int M : {-1, 0, 1, 64, 128, 129, 257, 1024, 2048, 2049, LORA_MAX_ROWS, LORA_MAX_ROWS + 1})
            for (int d : {-16, 0, 8, 16, 120, 128, 4096, 4104, 11008, LORA_INT8_MAX_D_IN, 1 << 17, 1 << 20, INT_MAX})
                for (int n : {8, 12, 4104, 1 << 20})
                    for (int na : {0, 1, 256, LORA_MAX_ADAPTERS}) {
                        const size_t b = lora_int8_workspace_bytes(M, d, n, r, na);
                        const bool ok = r >= 1 && r <= 64 && M > 0 && M <= LORA_MAX_ROWS && d > 0 && d % 16 == 0 &&
                                        d <= LORA_INT8_MAX_D_IN && n % 8 == 0 && na >= 1;
                        if ((b != 0) != ok || b % 256 != 0) {
                            fprintf(stderr, "int8 workspace bytes %zu for M %d d %d x %d r %d n %d\n", b, M, d, n, r, na);
                            ++failures;
                        }
                    }
    const size_t ws = lora_int8_workspace_bytes(64, 4096, 4096, 16, 32);
    const auto run = [&](const lora_epilogue_t *e, int M, int d, const void *x8, const float *xs, lora_mode_t mode,
                         size_t nb) {
        return lora_linear_int8(x8, xs, F, FF, F, F, FF, nullptr, FI, M, d, 4096, 16, 32, nullptr, e, F, LORA_BF16,
                                mode, F, nb, nullptr);
    };
    const lora_mode_t any = LORA_MODE_AUTO;
    EXPECT(run(nullptr, 64, 4104, F, FF, any, ws), LORA_ERR_SHAPE);
    EXPECT(run(nullptr, 64, LORA_INT8_MAX_D_IN + 16, F, FF, any, ws), LORA_ERR_SHAPE);
    EXPECT(run(nullptr, 64, 4096, F, FF, LORA_MODE_DECODE, ws), LORA_ERR_MODE);
    EXPECT(run(nullptr, 64, 4096, nullptr, FF, any, ws), LORA_ERR_NULL);
    EXPECT(run(nullptr, 64, 4096, F, nullptr, any, ws), LORA_ERR_NULL);
    EXPECT(run(nullptr, 64, 4096, off(8), FF, any, ws), LORA_ERR_ALIGN);
    EXPECT(run(nullptr, 64, 4096, F, FF, any, ws - 1), LORA_ERR_WORKSPACE);
    const lora_epilogue_t bad{nullptr, nullptr, nullptr, static_cast<lora_act_t>(9)};
    EXPECT(run(&bad, 64, 4096, F, FF, any, ws), LORA_ERR_VALUE);
    EXPECT(run(nullptr, 0, 4096, nullptr, nullptr, any, 0), LORA_OK);
}

static void experts() {
    for (int M : {INT_MIN, -1, 0, 1, 128, 2048, 8192, 8193, INT_MAX})
        for (int k : {INT_MIN, 0, 1, 4, 64, 65, INT_MAX})
            for (int E : {0, 1, 32, 4096, 4097})
                for (int d : {-16, 112, 128, 136, 2880, 1 << 20, (1 << 20) + 16})
                    for (int ff : {120, 144, 2768, 1 << 20})
                        for (int r : {0, 4, 8, 24, 64, 72})
                            for (int na : {0, 1, 40, LORA_MAX_ADAPTERS, LORA_MAX_ADAPTERS + 1}) {
                                const size_t b = lora_moe_layer_workspace_bytes(M, k, E, d, ff, r, na);
                                const bool ok = M > 0 && k >= 1 && k <= 64 && (int64_t)M * k <= LORA_MOE_MAX_PAIRS &&
                                                E >= 1 && E <= 4096 && d >= 128 && d % 16 == 0 && d <= 1 << 20 &&
                                                ff >= 128 && ff % 16 == 0 && r >= 8 && r <= 64 && r % 8 == 0 &&
                                                na >= 1 && na <= LORA_MAX_ADAPTERS;
                                if ((b != 0) != ok || b % 256 != 0) {
                                    fprintf(stderr, "moe layer workspace bytes %zu for M %d k %d E %d d %d ff %d r %d n %d\n",
                                            b, M, k, E, d, ff, r, na);
                                    ++failures;
                                }
                            }
    const size_t ws = lora_moe_layer_workspace_bytes(64, 4, 32, 2880, 1440, 16, 8);
    lora_moe_weights_t w{{F, F, F}, {F, F, F}, {F, F, F}};
    const auto run = [&](const lora_moe_weights_t *wt, int M, const void *x, const void *res, int act, int mode,
                         size_t nb) {
        return lora_moe_layer(x, wt, FF, nullptr, FI, FI, nullptr, res, M, 4, 32, 2880, 1440, 16, 8,
                              static_cast<lora_act_t>(act), F, LORA_F32, static_cast<lora_mode_t>(mode), F, nb, nullptr);
    };
    EXPECT(run(&w, 2049, F, F, 0, 0, ws), LORA_ERR_SHAPE);
    EXPECT(run(&w, 64, F, F, 5, 0, ws), LORA_ERR_VALUE);
    EXPECT(run(&w, 64, F, F, 2, LORA_MODE_PREFILL, ws), LORA_ERR_MODE);
    EXPECT(run(nullptr, 64, F, F, 2, 0, ws), LORA_ERR_NULL);
    EXPECT(run(&w, 64, nullptr, F, 2, 0, ws), LORA_ERR_NULL);
    EXPECT(run(&w, 64, F, off(8), 2, 0, ws), LORA_ERR_ALIGN);
    EXPECT(run(&w, 64, F, F, 2, 0, ws - 1), LORA_ERR_WORKSPACE);
    for (lora_moe_proj_t *p : {&w.gate, &w.up, &w.down})
        for (const void **q : {&p->W, &p->A, &p->B}) {
            *q = nullptr;
            EXPECT(run(&w, 64, F, F, 2, 0, ws), LORA_ERR_NULL);
            *q = off(8);
            EXPECT(run(&w, 64, F, F, 2, 0, ws), LORA_ERR_ALIGN);
            *q = F;
        }
    EXPECT(run(nullptr, 0, nullptr, nullptr, 2, 0, 0), LORA_OK);
}

static void rope() {
    const double *const D = static_cast<const double *>(F);
    const auto run = [&](int M, int qh, int kh, int hd, int rd, int64_t qs, int64_t ks, int layout, float f, int inv,
                         const void *q, int dtype) {
        return lora_rope(q, F, FI, D, M, qh, kh, hd, rd, qs, ks, static_cast<lora_rope_t>(layout), f, inv, off(1 << 16),
                         qs, off(1 << 16), ks, static_cast<lora_dtype_t>(dtype), nullptr);
    };
    const int64_t big = LORA_ROPE_MAX_STRIDE;
    EXPECT(run(0, 1024, 1024, 1024, 1024, big, big, 0, 1.0f, 0, nullptr, 0), LORA_OK);
    for (int M : {INT_MIN, -1, LORA_MAX_ROWS + 1, INT_MAX})
        EXPECT(run(M, 8, 2, 64, 64, 512, 128, 0, 1.0f, 0, F, 0), LORA_ERR_SHAPE);
    for (int h : {INT_MIN, 0, 1025, INT_MAX}) EXPECT(run(4, h, 2, 64, 64, big, 128, 0, 1.0f, 0, F, 0), LORA_ERR_SHAPE);
    for (int h : {INT_MIN, -1, 1025, INT_MAX}) EXPECT(run(4, 8, h, 64, 64, big, big, 0, 1.0f, 0, F, 0), LORA_ERR_SHAPE);
    for (int d : {INT_MIN, 0, 4, 12, 1032, INT_MAX}) EXPECT(run(4, 8, 2, d, 2, big, big, 0, 1.0f, 0, F, 0), LORA_ERR_SHAPE);
    for (int r : {INT_MIN, 0, 1, 63, 66, INT_MAX}) EXPECT(run(4, 8, 2, 64, r, 512, 128, 0, 1.0f, 0, F, 0), LORA_ERR_SHAPE);
    for (int64_t s : {INT64_MIN, (int64_t)-512, (int64_t)504, (int64_t)513, big + 8, INT64_MAX})
        EXPECT(run(4, 8, 2, 64, 64, s, 128, 0, 1.0f, 0, F, 0), LORA_ERR_SHAPE);
    EXPECT(run(4, 8, 2, 64, 64, 512, 128, 2, 1.0f, 0, F, 0), LORA_ERR_MODE);
    EXPECT(run(4, 8, 2, 64, 64, 512, 128, 0, 1.0f, 0, F, 2), LORA_ERR_DTYPE);
    for (float f : {0.0f, -1.0f, INFINITY, NAN}) EXPECT(run(4, 8, 2, 64, 64, 512, 128, 0, f, 0, F, 0), LORA_ERR_VALUE);
    EXPECT(run(4, 8, 2, 64, 64, 512, 128, 0, 1.0f, 2, F, 0), LORA_ERR_VALUE);
    EXPECT(run(4, 8, 2, 64, 64, 512, 128, 0, 1.0f, 0, nullptr, 0), LORA_ERR_NULL);
    EXPECT(run(4, 8, 2, 64, 64, 512, 128, 0, 1.0f, 0, off(2), 0), LORA_ERR_ALIGN);

    double table[LORA_ROPE_MAX_DIM / 2];
    float factor;
    for (int r : {2, 4, 62, 64, 128, LORA_ROPE_MAX_DIM})
        for (int s = 0; s <= 3; ++s)
            for (double stretch : {1.0, 8.0, 1e300}) {
                EXPECT(lora_rope_freqs(r, 1e4, static_cast<lora_rope_scaling_t>(s), stretch, 4096.0, table, &factor), LORA_OK);
                for (int i = 0; i < r / 2; ++i)
                    if (!(table[i] >= 0.0 && table[i] < 0.2)) ++failures;
                if (!(factor >= 1.0f && factor < 100.0f)) ++failures;
            }
    for (int r : {INT_MIN, 0, 1, 63, LORA_ROPE_MAX_DIM + 2, INT_MAX})
        EXPECT(lora_rope_freqs(r, 1e4, LORA_ROPE_PLAIN, 1.0, 1.0, table, &factor), LORA_ERR_SHAPE);
    EXPECT(lora_rope_freqs(64, 1e4, static_cast<lora_rope_scaling_t>(4), 1.0, 1.0, table, &factor), LORA_ERR_MODE);
    EXPECT(lora_rope_freqs(64, 1.0, LORA_ROPE_PLAIN, 1.0, 1.0, table, &factor), LORA_ERR_VALUE);
    EXPECT(lora_rope_freqs(64, 1e4, LORA_ROPE_LINEAR, 0.0, 1.0, table, &factor), LORA_ERR_VALUE);
    EXPECT(lora_rope_freqs(64, 1e4, LORA_ROPE_YARN, 2.0, NAN, table, &factor), LORA_ERR_VALUE);
    EXPECT(lora_rope_freqs(64, 1e4, LORA_ROPE_YARN, 2.0, 1.0, nullptr, &factor), LORA_ERR_NULL);
    EXPECT(lora_rope_freqs(64, 1e4, LORA_ROPE_YARN, 2.0, 1.0, table, nullptr), LORA_ERR_NULL);
}

int main() {
    rows();
    layer();
    experts();
    rope();
    if (failures) {
        fprintf(stderr, "%d unexpected results\n", failures);
        return 1;
    }
    printf("abi driver: all calls returned the expected status\n");
    return 0;
}
