/* host_checks_w8a8.c -- test infrastructure: the host-side argument checks of
 * the W8A8 and router-balance entry points, for an AddressSanitizer /
 * UndefinedBehaviorSanitizer build of the library's host code
 * (tests/test_sanitizers_w8a8.py), at the smallest and largest sizes.  Every
 * call is rejected by the checks or has nothing to do, so nothing reaches the
 * HIP runtime: the device pointers are placeholders that are never
 * dereferenced.  Exit status 0 when every call returned the documented status. */
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "moe_w4a16.h"

static int fails = 0;
#define EXPECT(call, want)                                                                    \
    do {                                                                                      \
        moe_status got_ = (call);                                                             \
        if (got_ != (want)) {                                                                 \
            printf("line %d: %s returned %d (%s), expected %d\n", __LINE__, #call, (int)got_, \
                   moe_status_str(got_), (int)(want));                                        \
            ++fails;                                                                          \
        }                                                                                     \
    } while (0)
#define SIZE(call, want)                                                                                \
    do {                                                                                                \
        size_t got_ = (call);                                                                           \
        if (got_ != (size_t)(want)) {                                                                   \
            printf("line %d: %s is %zu, expected %zu\n", __LINE__, #call, got_, (size_t)(want));        \
            ++fails;                                                                                    \
        }                                                                                               \
    } while (0)

int main(void) {
    void *P = (void *)(uintptr_t)0x10000, *U = (void *)(uintptr_t)0x10002;
    const uint16_t *x = P;
    int8_t *c = P;
    uint8_t *u8 = P;
    float *f = P;
    int32_t *i = P;
    uint16_t *o = P;
    const int32_t most = 1 << 20;  /* MOE_MAX_TOKENS */
    const int32_t wrong[] = {INT32_MIN, -1, 8, 17, 65552, INT32_MAX};

    moe_layer_desc d;
    memset(&d, 0, sizeof d);
    d.hidden = 4096; d.inter = 2048; d.n_routed = 256; d.top_k = 8; d.n_shared = 1; d.group_size = 128;
    d.routed_scale = 1.0f;
    moe_layer_desc bad = d;
    bad.n_routed = 257;

    for (unsigned s = 0; s < sizeof wrong / sizeof *wrong; ++s) {
        const int32_t n = wrong[s];
        EXPECT(moe_act_quant_int8(1, n, x, c, f, NULL), MOE_ERR_SHAPE);
        EXPECT(moe_w8a8_prepack(1, n, 64, c, c, NULL), MOE_ERR_SHAPE);
        EXPECT(moe_w8a8_prepack(1, 64, n, c, c, NULL), MOE_ERR_SHAPE);
        SIZE(moe_w8a8_packed_bytes(1, n, 64), 0);
        SIZE(moe_w8a8_packed_bytes(1, 64, n), 0);
        EXPECT(moe_w8a8_gemm(most, n, 64, c, f, c, f, o, NULL), MOE_ERR_SHAPE);
        EXPECT(moe_w8a8_gemm(most, 64, n, c, f, c, f, o, NULL), MOE_ERR_SHAPE);
        EXPECT(moe_w8a8_linear(most, n, 64, x, c, f, c, f, o, NULL), MOE_ERR_SHAPE);
        EXPECT(moe_w8a8_linear(most, 64, n, x, c, f, c, f, o, NULL), MOE_ERR_SHAPE);
        EXPECT(moe_w8a8_grouped_gemm(&d, most, c, f, i, most, n, 64, c, f, i, 0, o, NULL), MOE_ERR_SHAPE);
        EXPECT(moe_w8a8_grouped_gemm(&d, most, c, f, i, most, 64, n, c, f, i, 0, o, NULL), MOE_ERR_SHAPE);
    }
    const int32_t counts[] = {INT32_MIN, -1, most + 1, INT32_MAX};
    for (unsigned s = 0; s < sizeof counts / sizeof *counts; ++s) {
        const int32_t n = counts[s];
        EXPECT(moe_w8a8_gemm(n, 64, 64, c, f, c, f, o, NULL), MOE_ERR_SHAPE);
        EXPECT(moe_w8a8_linear(n, 64, 64, x, c, f, c, f, o, NULL), MOE_ERR_SHAPE);
        EXPECT(moe_w8a8_grouped_gemm(&d, n, c, f, i, 1, 128, 64, c, f, i, 1, o, NULL), MOE_ERR_SHAPE);
        EXPECT(moe_w8a8_grouped_gemm(&d, 1, c, f, i, n, 128, 64, c, f, i, 1, o, NULL), MOE_ERR_SHAPE);
        EXPECT(moe_w8a8_experts(&d, n, x, f, i, i, i, c, f, c, f, c, f, o, c, f, o, o, NULL), MOE_ERR_SHAPE);
        EXPECT(moe_balance_loss(&d, n, 1, i, u8, f, i, 0.1f, i, f, f, f, P, 1 << 30, NULL), MOE_ERR_SHAPE);
        EXPECT(moe_balance_loss(&d, 1, n, i, u8, f, i, 0.1f, i, f, f, f, P, 1 << 30, NULL), MOE_ERR_SHAPE);
        EXPECT(moe_route_backward(&d, n, 1, i, u8, f, i, i, f, f, f, f, NULL), MOE_ERR_SHAPE);
        EXPECT(moe_route_backward(&d, 1, n, i, u8, f, i, i, f, f, f, f, NULL), MOE_ERR_SHAPE);
        SIZE(moe_balance_workspace_bytes(&d, n, 1), 0);
        SIZE(moe_balance_workspace_bytes(&d, 1, n), 0);
        SIZE(moe_w8a8_packed_bytes(n, 64, 64), 0);
    }
    EXPECT(moe_act_quant_int8(most * 9 + 1, 64, x, c, f, NULL), MOE_ERR_SHAPE);
    EXPECT(moe_act_quant_int8(INT32_MIN, 64, x, c, f, NULL), MOE_ERR_SHAPE);
    EXPECT(moe_act_quant_int8(most * 9, 65536, U, c, f, NULL), MOE_ERR_ALIGN);
    EXPECT(moe_w8a8_prepack(257, 65536, 65536, c, U, NULL), MOE_ERR_ALIGN);
    EXPECT(moe_w8a8_prepack(257, 65536, 65536, c, c + 16, NULL), MOE_ERR_SHAPE);  /* overlapping */
    EXPECT(moe_w8a8_gemm(most, 65536, 65536, U, f, c, f, o, NULL), MOE_ERR_ALIGN);
    EXPECT(moe_w8a8_linear(most, 65536, 65536, U, c, f, c, f, o, NULL), MOE_ERR_ALIGN);
    EXPECT(moe_w8a8_grouped_gemm(&d, most, c, f, i, most, 65536, 65536, c, f, i, 1, U, NULL), MOE_ERR_ALIGN);
    EXPECT(moe_w8a8_grouped_gemm(&d, most, c, f, i, most, 128, 64, c, f, i, 2, o, NULL), MOE_ERR_UNSUPPORTED);
    EXPECT(moe_w8a8_grouped_gemm(&bad, 1, c, f, i, 1, 128, 64, c, f, i, 1, o, NULL), MOE_ERR_SHAPE);
    EXPECT(moe_w8a8_grouped_gemm(NULL, 1, c, f, i, 1, 128, 64, c, f, i, 1, o, NULL), MOE_ERR_NULL);
    EXPECT(moe_w8a8_experts(&d, most, U, f, i, i, i, c, f, c, f, c, f, o, c, f, o, o, NULL), MOE_ERR_ALIGN);
    EXPECT(moe_w8a8_experts(&bad, 1, x, f, i, i, i, c, f, c, f, c, f, o, c, f, o, o, NULL), MOE_ERR_SHAPE);
    EXPECT(moe_balance_loss(&d, most, most, NULL, NULL, f, i, 0.1f, i, f, f, f, P, 1 << 30, NULL), MOE_ERR_NULL);
    EXPECT(moe_balance_loss(&d, most, most, i, NULL, f, i, 0.1f, i, f, f, f, P, 1 << 20, NULL), MOE_ERR_WORKSPACE);
    EXPECT(moe_balance_loss(&d, most, 1, i, NULL, f, i, 0.1f, i, f, f, f, P, 0, NULL), MOE_ERR_WORKSPACE);
    EXPECT(moe_balance_loss(&bad, 1, 1, i, NULL, f, i, 0.1f, i, f, f, f, P, 1 << 20, NULL), MOE_ERR_SHAPE);
    EXPECT(moe_route_backward(&d, most, most, NULL, NULL, f, i, i, f, f, f, f, NULL), MOE_ERR_NULL);
    EXPECT(moe_route_backward(&d, most, 1, NULL, NULL, f, i, NULL, f, f, f, f, NULL), MOE_ERR_NULL);
    EXPECT(moe_route_backward(&bad, 1, 1, NULL, NULL, f, i, i, f, f, f, f, NULL), MOE_ERR_SHAPE);

    /* nothing to do */
    EXPECT(moe_act_quant_int8(0, 65536, NULL, NULL, NULL, NULL), MOE_OK);
    EXPECT(moe_w8a8_gemm(0, 65536, 65536, NULL, NULL, NULL, NULL, NULL, NULL), MOE_OK);
    EXPECT(moe_w8a8_linear(0, 16, 16, NULL, NULL, NULL, NULL, NULL, NULL, NULL), MOE_OK);
    EXPECT(moe_w8a8_grouped_gemm(&d, 0, NULL, NULL, NULL, 0, 128, 16, NULL, NULL, NULL, 1, NULL, NULL), MOE_OK);
    EXPECT(moe_route_backward(&d, 0, 1, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL), MOE_OK);

    /* sizes: 64 bytes, a double per sequence and 64 experts, 256 sums and counts and a token count per chunk of tokens
       and sequence, a token count per sequence; rounded up to 256 */
    SIZE(moe_w8a8_packed_bytes(257, 65536, 65536), (size_t)257 << 32);
    SIZE(moe_balance_workspace_bytes(&d, 0, 1), (64 + 32 + 2052 + 4 + 255) / 256 * 256);
    SIZE(moe_balance_workspace_bytes(&d, most, most),
         ((size_t)64 + 32 * (size_t)most + 2052 * (size_t)(8192 + most) + 4 * (size_t)most + 255) / 256 * 256);

    printf("host checks: %d failures\n", fails);
    return fails ? 1 : 0;
}
