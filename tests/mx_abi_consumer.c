/* A C program against the microscaled calls of include/razer.h: sizes, and
 * the documented statuses of calls that are refused before any launch. */
#include <stdio.h>

#include "razer.h"

#define CHECK(cond)                                             \
    do {                                                        \
        if (!(cond)) {                                          \
            fprintf(stderr, "line %d: %s\n", __LINE__, #cond);  \
            return 1;                                           \
        }                                                       \
    } while (0)

int main(void)
{
    static _Alignas(16) uint8_t buf[64];
    static _Alignas(16) int32_t off[4];
    float ts = 1.0f;
    CHECK(razer_scale_tiles_size(RAZER_FMT_MXFP4, 129, 256, 0) == 2 * 2 * 512);
    CHECK(razer_scale_tiles_size(RAZER_FMT_NVFP4, 129, 256, 3) == 4 * 4 * 512);
    CHECK(razer_workspace_size(RAZER_OP_GEMM_MX_ONLINE, 16, 64, 256) == 0);
    CHECK(razer_workspace_size(RAZER_OP_GEMM_MX_ONLINE, 32, 64, 256) == 32 * 128 + 2 * 512);
    CHECK(razer_gemm_mx_grouped_workspace_size(256, 256, 2) == 256 * 128 + 4 * 2 * 512);
    CHECK(razer_quantize_mx(buf, RAZER_F32, 1, 32, NULL, 0, buf, buf, NULL) == RAZER_ERR_DTYPE);
    CHECK(razer_quantize_mx(buf, RAZER_BF16, 1, 40, NULL, 0, buf, buf, NULL) == RAZER_ERR_SHAPE);
    CHECK(razer_quantize_mx(buf, RAZER_BF16, 0, 32, NULL, 0, NULL, NULL, NULL) == RAZER_OK);
    CHECK(razer_dequant_mx(buf + 1, buf, 1, 32, NULL, 0, buf, RAZER_F16, NULL) == RAZER_ERR_ALIGN);
    CHECK(razer_tile_scales(buf, 2, 1, 4, off, 2, buf, NULL) == RAZER_ERR_SHAPE);
    CHECK(razer_gemm_mx(buf, buf, NULL, 1, buf, buf, NULL, RAZER_FMT_NVFP4, 1, 32, RAZER_ACT_NONE, buf, RAZER_BF16, NULL) == RAZER_ERR_INVALID_ARG);
    CHECK(razer_gemm_mx(buf, buf, &ts, 1, buf, buf, &ts, RAZER_FMT_WEIGHT, 1, 32, RAZER_ACT_NONE, buf, RAZER_BF16, NULL) == RAZER_ERR_UNSUPPORTED);
    CHECK(razer_gemm_mx_grouped(buf, buf, NULL, 1, NULL, 1, buf, buf, NULL, RAZER_FMT_MXFP4, 2, 32, RAZER_ACT_SILU_MUL, buf, RAZER_BF16, NULL) ==
          RAZER_ERR_INVALID_ARG);
    CHECK(razer_gemm_mx_online(buf, RAZER_F16, 32, buf, buf, 1, 32, RAZER_ACT_SILU_MUL, buf, RAZER_BF16, NULL, 0, NULL) == RAZER_ERR_SHAPE);
    CHECK(razer_gemm_mx_grouped_online(buf, RAZER_F16, 64, off, 1, buf, buf, 1, 32, RAZER_ACT_NONE, buf, RAZER_BF16, NULL, 0, NULL) ==
          RAZER_ERR_WORKSPACE);
    puts("all checks passed");
    return 0;
}
