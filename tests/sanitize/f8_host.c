/*
 * Drives the host side of the 8-bit floating point and checkpoint calls
 * (include/rbq.h) so that it can run under AddressSanitizer and
 * UndefinedBehaviorSanitizer: workspace sizes and tile plans over ordinary
 * and extreme shapes, limits, and argument checks.  No call here reaches a
 * device; the pointers are aligned stand-in addresses that the checks compare
 * but never dereference.
 * Test infrastructure: built and run by tests/test_sanitizers_f8_cpu.py.
 */
#include <stdint.h>
#include <stdio.h>

#include "rbq.h"

static int failures = 0;
#define CHECK(cond)                                                     \
    do {                                                                \
        if (!(cond)) {                                                  \
            fprintf(stderr, "FAIL %s:%d: %s\n", __FILE__, __LINE__, #cond); \
            ++failures;                                                 \
        }                                                               \
    } while (0)

static void *buf(int k) { return (void *)(((uintptr_t)1 << 30) + (uintptr_t)k * ((uintptr_t)1 << 20)); }
static void *odd(int k) { return (void *)((uintptr_t)buf(k) + 1); }

static const int32_t OUTS[] = {1, 15, 16, 127, 128, 129, 600, 4096, 5003, 11008, 1 << 20, RBQ_F8_MAX_FEATURES};
static const int32_t INS[] = {32, 96, 128, 160, 4096, 4128, 14336, 1 << 20, RBQ_F8_MAX_FEATURES};
static const int32_t TOKENS[] = {1, 16, 17, 32, 33, 64, 65, 128, 129, 300, 2048, 100000, 1 << 24, 0x7FFFFFFF};
#define N(a) (sizeof(a) / sizeof((a)[0]))

static void sizes(void)
{
    for (size_t o = 0; o < N(OUTS); ++o)
        for (size_t i = 0; i < N(INS); ++i)
            for (size_t m = 0; m < N(TOKENS); ++m) {
                const uint64_t out = (uint64_t)OUTS[o], in = (uint64_t)INS[i], M = (uint64_t)TOKENS[m];
                for (int y = 0; y <= 1; ++y) {
                    const size_t n = rbq_gemm_f8_workspace_bytes(OUTS[o], INS[i], TOKENS[m], y);
                    CHECK(n % 16 == 0);
                    CHECK(n <= 34 * ((M + 255) / 256 * 256) * ((out + 127) / 128 * 128));
                    CHECK(M > 32 || n == 0);
                }
                for (int K = 1; K <= 4; ++K)
                    for (int g = 0; g <= 128; g += 128) {
                        const rbq_shape s = {OUTS[o], INS[i], K, g};
                        const size_t n = rbq_qat_backward_ckpt_workspace_bytes(s, TOKENS[m]);
                        if (g != 0 && in % 128 != 0)
                            CHECK(n == 0);
                        CHECK(n <= 4 * (8 * out * in + 8 * (uint64_t)K * out * (in / 128 + 1) + 32 * M * in));
                    }
            }
    CHECK(rbq_gemm_f8_workspace_bytes(0, 64, 64, 0) == 0);
    CHECK(rbq_gemm_f8_workspace_bytes(64, 0, 64, 0) == 0);
    CHECK(rbq_gemm_f8_workspace_bytes(64, 64, 0, 0) == 0);
    CHECK(rbq_gemm_f8_workspace_bytes(-1, 64, 64, 0) == 0);
    CHECK(rbq_gemm_f8_workspace_bytes(64, 64, 64, 2) == 0);
    CHECK(rbq_gemm_f8_workspace_bytes(INT32_MAX, INT32_MAX, INT32_MAX, 0) == 0);
    CHECK(rbq_gemm_f8_workspace_bytes(INT32_MIN, INT32_MIN, INT32_MIN, INT32_MIN) == 0);
    const rbq_shape extreme[] = {{INT32_MAX, INT32_MAX - 31, 2, 0}, {INT32_MIN, INT32_MIN, INT32_MIN, INT32_MIN},
                                 {0, 0, 0, 0}, {64, 64, 5, 0}, {64, 64, 2, 64}, {64, 48, 2, 0}};
    for (size_t i = 0; i < N(extreme); ++i)
        for (size_t m = 0; m < N(TOKENS); ++m)
            CHECK(rbq_qat_backward_ckpt_workspace_bytes(extreme[i], TOKENS[m]) == 0);
}

static void arguments(void)
{
    const int32_t wild[] = {INT32_MIN, -1, 31, 33, INT32_MAX};
    for (size_t i = 0; i < N(wild); ++i) {
        const int32_t n = wild[i];
        CHECK(rbq_encode_f8(buf(0), 64, n, buf(1), buf(2), NULL, NULL) == RBQ_ERR_INVALID_ARG);
        CHECK(rbq_quantize_f8(buf(0), 4, n, buf(1), buf(2), NULL) == RBQ_ERR_INVALID_ARG);
        CHECK(rbq_gemm_f8(buf(0), buf(1), 64, n, buf(2), buf(3), 4, buf(4), 0, NULL, 0, NULL) == RBQ_ERR_INVALID_ARG);
        CHECK(rbq_gemv_f8(buf(0), buf(1), 64, n, buf(2), buf(3), NULL) == RBQ_ERR_INVALID_ARG);
        CHECK(rbq_qat_checkpoint(buf(0), 4, n, buf(1), buf(2), NULL) == RBQ_ERR_INVALID_ARG);
    }
    CHECK(rbq_encode_f8(buf(0), INT32_MAX, 64, buf(1), buf(2), NULL, NULL) == RBQ_ERR_UNSUPPORTED);
    CHECK(rbq_encode_f8(buf(0), INT32_MIN, 64, buf(1), buf(2), NULL, NULL) == RBQ_ERR_INVALID_ARG);
    CHECK(rbq_encode_f8(odd(0), 64, 64, buf(1), buf(2), NULL, NULL) == RBQ_ERR_ALIGNMENT);
    CHECK(rbq_encode_f8(NULL, 64, 64, buf(1), buf(2), NULL, NULL) == RBQ_ERR_INVALID_ARG);
    CHECK(rbq_quantize_f8(buf(0), INT32_MIN, 64, buf(1), buf(2), NULL) == RBQ_ERR_INVALID_ARG);
    CHECK(rbq_quantize_f8(buf(0), 4, INT32_MAX - 31, buf(1), buf(2), NULL) == RBQ_ERR_UNSUPPORTED);
    CHECK(rbq_quantize_f8(buf(0), 4, 64, odd(1), buf(2), NULL) == RBQ_ERR_ALIGNMENT);
    CHECK(rbq_gemm_f8(buf(0), buf(1), 64, 64, buf(2), buf(3), 4, buf(4), 2, NULL, 0, NULL) == RBQ_ERR_INVALID_ARG);
    CHECK(rbq_gemm_f8(buf(0), buf(1), 64, 64, buf(2), buf(3), 4, buf(4), 0, NULL, 4, NULL) == RBQ_ERR_INVALID_ARG);
    CHECK(rbq_gemm_f8(buf(0), buf(1), 64, 64, buf(2), buf(3), 4, odd(4), 0, NULL, 0, NULL) == RBQ_ERR_ALIGNMENT);
    CHECK(rbq_gemv_f8(buf(0), buf(1), 64, 64, odd(2), buf(3), NULL) == RBQ_ERR_ALIGNMENT);
    CHECK(rbq_gemv_f8(buf(0), NULL, 64, 64, buf(2), buf(3), NULL) == RBQ_ERR_INVALID_ARG);
    CHECK(rbq_qat_checkpoint(buf(0), 4, 64, buf(1), odd(2), NULL) == RBQ_ERR_ALIGNMENT);
    CHECK(rbq_qat_checkpoint(NULL, 4, 64, buf(1), buf(2), NULL) == RBQ_ERR_INVALID_ARG);
    const rbq_shape s = {64, 256, 2, 0};
    CHECK(rbq_qat_backward_ckpt(buf(0), buf(1), s, buf(2), buf(3), buf(4), INT32_MIN, buf(5), buf(6), buf(7), NULL, 0,
                                NULL, NULL) == RBQ_ERR_INVALID_ARG);
    CHECK(rbq_qat_backward_ckpt(buf(0), buf(1), s, buf(2), buf(3), buf(4), 4, buf(5), NULL, buf(7), NULL, 0, NULL,
                                NULL) == RBQ_ERR_INVALID_ARG);
    CHECK(rbq_qat_backward_ckpt(buf(0), buf(1), s, odd(2), buf(3), buf(4), 4, buf(5), buf(6), buf(7), NULL, 0, NULL,
                                NULL) == RBQ_ERR_ALIGNMENT);
    /* nothing to do: no device is looked for */
    CHECK(rbq_encode_f8(NULL, 0, 64, NULL, NULL, NULL, NULL) == RBQ_OK);
    CHECK(rbq_quantize_f8(NULL, 0, 64, NULL, NULL, NULL) == RBQ_OK);
    CHECK(rbq_gemm_f8(NULL, NULL, 64, 64, NULL, NULL, 0, NULL, 0, NULL, 0, NULL) == RBQ_OK);
    CHECK(rbq_gemv_f8(NULL, NULL, 0, 64, NULL, NULL, NULL) == RBQ_OK);
    CHECK(rbq_qat_checkpoint(NULL, 0, 64, NULL, NULL, NULL) == RBQ_OK);
}

int main(void)
{
    sizes();
    arguments();
    if (failures != 0) {
        fprintf(stderr, "%d checks failed\n", failures);
        return 1;
    }
    puts("8-bit host checks passed");
    return 0;
}
