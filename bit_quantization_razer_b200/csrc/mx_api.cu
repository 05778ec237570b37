// extern "C" surface of the microscaled 4-bit operators (mx.cu, mx_gemm.cu):
// argument checks, then the launches.  No call allocates or synchronises.
#include "mx.cuh"

namespace razer {

razer_status run_quantize_mx(const void *X, razer_dtype dt, int64_t M, int64_t K, const int32_t *offsets, int E, uint8_t *codes,
                             uint8_t *tiles, cudaStream_t st);
razer_status run_dequant_mx(const uint8_t *codes, const uint8_t *tiles, int64_t M, int64_t K, const int32_t *offsets, int E, void *out,
                            razer_dtype dt, cudaStream_t st);
razer_status run_tile_scales(const uint8_t *rows, int64_t batch, int64_t R, int64_t C, const int32_t *offsets, int E, uint8_t *tiles,
                             cudaStream_t st);
bool gemm_mx_fuses(int64_t T, int64_t E);
razer_status run_gemm_mx(const void *X, razer_dtype x_dt, const uint8_t *codes_a, const uint8_t *tiles_a, const float *ts_a, int64_t T, const int32_t *offsets, int E,
                         const uint8_t *codes_w, const uint8_t *tiles_w, const float *ts_w, razer_format fmt, int64_t N, int64_t K, int gate,
                         void *Y, razer_dtype out_dt, cudaStream_t st);

static bool int32_size(int64_t v) { return v >= 0 && v <= INT32_MAX; }

// sizes and groups shared by every call: rows T in E groups (E = 0: dense)
static razer_status check_rows(int64_t T, int64_t K, const int32_t *offsets, int64_t E)
{
    if (!int32_size(T) || !int32_size(K) || K % 32 != 0 || !int32_size(E)) return RAZER_ERR_SHAPE;
    if (E > 0 && !offsets) return RAZER_ERR_INVALID_ARG;
    if (E > 0 && !aligned(offsets, 4)) return RAZER_ERR_ALIGN;
    return RAZER_OK;
}

// the weights and the output of a product; gate != 0: N counts gate and up rows
static razer_status check_product(int64_t T, int64_t N, int64_t K, int64_t E, const uint8_t *codes_w, const uint8_t *scales_w,
                                  const float *ts_w, razer_act act, const void *Y, razer_dtype out_dt)
{
    if (act != RAZER_ACT_NONE && act != RAZER_ACT_SILU_MUL) return RAZER_ERR_INVALID_ARG;
    if (!valid_dt(out_dt)) return RAZER_ERR_INVALID_ARG;
    if (!int32_size(N) || (act == RAZER_ACT_SILU_MUL && N % 2 != 0)) return RAZER_ERR_SHAPE;
    if (E > 0 && N > INT32_MAX / E) return RAZER_ERR_SHAPE;
    if (T * N > 0 && !Y) return RAZER_ERR_INVALID_ARG;
    if (N * K > 0 && (!codes_w || !scales_w)) return RAZER_ERR_INVALID_ARG;
    if (!aligned(codes_w, 16) || !aligned(scales_w, 16) || !aligned(ts_w, 4) || !aligned(Y, 16)) return RAZER_ERR_ALIGN;
    return RAZER_OK;
}

static size_t packed_bytes(int64_t T, int64_t K) { return ((size_t)T * (size_t)K / 2 + 255) & ~(size_t)255; }

static size_t mx_tiles_bytes(bool nv, int64_t T, int64_t K, int64_t E)
{
    const int64_t rows = E > 0 ? mx::tile_rows_grouped(T, E) : mx::tile_rows(T);
    return (size_t)rows * (size_t)mx::tile_cols(nv, K) * mx::kTileBytes;
}

size_t gemm_mx_online_workspace_bytes(int64_t T, int64_t K, int64_t E)
{
    if (T <= 0 || K <= 0 || E < 0 || gemm_mx_fuses(T, E)) return 0;
    return packed_bytes(T, K) + mx_tiles_bytes(false, T, K, E);
}

static razer_status gemm_mx_checked(const uint8_t *codes_a, const uint8_t *scales_a, const float *ts_a, int64_t T, const int32_t *offsets,
                                    int64_t E, const uint8_t *codes_w, const uint8_t *scales_w, const float *ts_w, razer_format fmt,
                                    int64_t N, int64_t K, razer_act act, void *Y, razer_dtype out_dt, cudaStream_t st)
{
    if (fmt != RAZER_FMT_MXFP4 && fmt != RAZER_FMT_NVFP4) return valid_fmt(fmt) ? RAZER_ERR_UNSUPPORTED : RAZER_ERR_INVALID_ARG;
    razer_status s = check_rows(T, K, offsets, E);
    if (s != RAZER_OK) return s;
    if ((s = check_product(T, N, K, E, codes_w, scales_w, ts_w, act, Y, out_dt)) != RAZER_OK) return s;
    if (T * K > 0 && (!codes_a || !scales_a)) return RAZER_ERR_INVALID_ARG;
    if (!aligned(codes_a, 16) || !aligned(scales_a, 16) || !aligned(ts_a, 4)) return RAZER_ERR_ALIGN;
    // NVFP4 values are code * scale * ts: without ts the call is incomplete
    if (fmt == RAZER_FMT_NVFP4 && (!ts_a || !ts_w)) return RAZER_ERR_INVALID_ARG;
    if (T == 0 || N == 0) return RAZER_OK;
    return run_gemm_mx(nullptr, RAZER_BF16, codes_a, scales_a, ts_a, T, offsets, (int)E, codes_w, scales_w, ts_w, fmt, N, K, act == RAZER_ACT_SILU_MUL ? 1 : 0, Y,
                       out_dt, st);
}

static razer_status gemm_mx_online_checked(const void *X, razer_dtype x_dt, int64_t T, const int32_t *offsets, int64_t E,
                                           const uint8_t *codes_w, const uint8_t *scales_w, int64_t N, int64_t K, razer_act act, void *Y,
                                           razer_dtype out_dt, void *workspace, size_t ws_bytes, cudaStream_t st)
{
    razer_status s = check_rows(T, K, offsets, E);
    if (s != RAZER_OK) return s;
    if ((s = check_product(T, N, K, E, codes_w, scales_w, nullptr, act, Y, out_dt)) != RAZER_OK) return s;
    if (!valid_dt(x_dt)) return RAZER_ERR_INVALID_ARG;
    if (!in16(x_dt)) return RAZER_ERR_DTYPE;
    if (T * K > 0 && !X) return RAZER_ERR_INVALID_ARG;
    if (!aligned(X, 16)) return RAZER_ERR_ALIGN;
    if (T == 0 || N == 0) return RAZER_OK;
    const size_t need = gemm_mx_online_workspace_bytes(T, K, E);
    if (need) {
        if (!workspace || ws_bytes < need) return RAZER_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return RAZER_ERR_ALIGN;
    }
    const int gate = act == RAZER_ACT_SILU_MUL ? 1 : 0;
    if (gemm_mx_fuses(T, E))
        return run_gemm_mx(X, x_dt, nullptr, nullptr, nullptr, T, offsets, (int)E, codes_w, scales_w, nullptr, RAZER_FMT_MXFP4, N, K, gate, Y, out_dt,
                           st);
    uint8_t *codes_a = reinterpret_cast<uint8_t *>(workspace), *scales_a = codes_a + packed_bytes(T, K);
    if (K > 0 && (s = run_quantize_mx(X, x_dt, T, K, offsets, (int)E, codes_a, scales_a, st)) != RAZER_OK) return s;
    return run_gemm_mx(nullptr, x_dt, codes_a, scales_a, nullptr, T, offsets, (int)E, codes_w, scales_w, nullptr, RAZER_FMT_MXFP4, N, K, gate, Y,
                       out_dt, st);
}

}  // namespace razer

using namespace razer;

extern "C" {

size_t razer_scale_tiles_size(razer_format fmt, int64_t R, int64_t K, int64_t E)
{
    if ((fmt != RAZER_FMT_MXFP4 && fmt != RAZER_FMT_NVFP4) || R < 0 || K < 0 || E < 0) return 0;
    return mx_tiles_bytes(fmt == RAZER_FMT_NVFP4, R, K, E);
}

razer_status razer_quantize_mx(const void *X, razer_dtype in_dt, int64_t M, int64_t K, const int32_t *offsets, int64_t E, uint8_t *codes,
                               uint8_t *scale_tiles, razer_stream_t stream)
{
    razer_status s = check_rows(M, K, offsets, E);
    if (s != RAZER_OK) return s;
    if (!valid_dt(in_dt)) return RAZER_ERR_INVALID_ARG;
    if (!in16(in_dt)) return RAZER_ERR_DTYPE;
    if (M * K == 0) return RAZER_OK;
    if (!X || !codes || !scale_tiles) return RAZER_ERR_INVALID_ARG;
    if (!aligned(X, 16) || !aligned(codes, 16) || !aligned(scale_tiles, 16)) return RAZER_ERR_ALIGN;
    return run_quantize_mx(X, in_dt, M, K, offsets, (int)E, codes, scale_tiles, (cudaStream_t)stream);
}

razer_status razer_dequant_mx(const uint8_t *codes, const uint8_t *scale_tiles, int64_t M, int64_t K, const int32_t *offsets, int64_t E,
                              void *out, razer_dtype out_dt, razer_stream_t stream)
{
    razer_status s = check_rows(M, K, offsets, E);
    if (s != RAZER_OK) return s;
    if (!valid_dt(out_dt)) return RAZER_ERR_INVALID_ARG;
    if (M * K == 0) return RAZER_OK;
    if (!codes || !scale_tiles || !out) return RAZER_ERR_INVALID_ARG;
    if (!aligned(codes, 16) || !aligned(scale_tiles, 16) || !aligned(out, 16)) return RAZER_ERR_ALIGN;
    return run_dequant_mx(codes, scale_tiles, M, K, offsets, (int)E, out, out_dt, (cudaStream_t)stream);
}

razer_status razer_tile_scales(const uint8_t *scales, int64_t batch, int64_t R, int64_t C, const int32_t *offsets, int64_t E,
                               uint8_t *scale_tiles, razer_stream_t stream)
{
    if (!int32_size(batch) || !int32_size(R) || !int32_size(C) || !int32_size(E)) return RAZER_ERR_SHAPE;
    if (E > 0 && batch != 1) return RAZER_ERR_SHAPE;
    if (E > 0 && !offsets) return RAZER_ERR_INVALID_ARG;
    if (E > 0 && !aligned(offsets, 4)) return RAZER_ERR_ALIGN;
    if (batch == 0 || R * C == 0) return RAZER_OK;
    const int64_t trows = E > 0 ? mx::tile_rows_grouped(R, E) : mx::tile_rows(R), chunks = (C + 15) / 16;
    if (trows > INT32_MAX / chunks || trows * chunks > INT32_MAX / batch) return RAZER_ERR_SHAPE;
    if (!scales || !scale_tiles) return RAZER_ERR_INVALID_ARG;
    if (!aligned(scale_tiles, 16)) return RAZER_ERR_ALIGN;
    return run_tile_scales(scales, batch, R, C, offsets, (int)E, scale_tiles, (cudaStream_t)stream);
}

razer_status razer_gemm_mx(const uint8_t *codes_a, const uint8_t *scales_a, const float *ts_a, int64_t M, const uint8_t *codes_w,
                           const uint8_t *scales_w, const float *ts_w, razer_format fmt, int64_t N, int64_t K, razer_act act, void *Y,
                           razer_dtype out_dt, razer_stream_t stream)
{
    return gemm_mx_checked(codes_a, scales_a, ts_a, M, nullptr, 0, codes_w, scales_w, ts_w, fmt, N, K, act, Y, out_dt, (cudaStream_t)stream);
}

razer_status razer_gemm_mx_grouped(const uint8_t *codes_a, const uint8_t *scales_a, const float *ts_a, int64_t T, const int32_t *offsets,
                                   int64_t E, const uint8_t *codes_w, const uint8_t *scales_w, const float *ts_w, razer_format fmt,
                                   int64_t N, int64_t K, razer_act act, void *Y, razer_dtype out_dt, razer_stream_t stream)
{
    if (E < 1) return RAZER_ERR_SHAPE;
    return gemm_mx_checked(codes_a, scales_a, ts_a, T, offsets, E, codes_w, scales_w, ts_w, fmt, N, K, act, Y, out_dt, (cudaStream_t)stream);
}

razer_status razer_gemm_mx_online(const void *X, razer_dtype x_dt, int64_t M, const uint8_t *codes_w, const uint8_t *scales_w, int64_t N,
                                  int64_t K, razer_act act, void *Y, razer_dtype out_dt, void *workspace, size_t ws_bytes,
                                  razer_stream_t stream)
{
    return gemm_mx_online_checked(X, x_dt, M, nullptr, 0, codes_w, scales_w, N, K, act, Y, out_dt, workspace, ws_bytes, (cudaStream_t)stream);
}

razer_status razer_gemm_mx_grouped_online(const void *X, razer_dtype x_dt, int64_t T, const int32_t *offsets, int64_t E,
                                          const uint8_t *codes_w, const uint8_t *scales_w, int64_t N, int64_t K, razer_act act, void *Y,
                                          razer_dtype out_dt, void *workspace, size_t ws_bytes, razer_stream_t stream)
{
    if (E < 1) return RAZER_ERR_SHAPE;
    return gemm_mx_online_checked(X, x_dt, T, offsets, E, codes_w, scales_w, N, K, act, Y, out_dt, workspace, ws_bytes, (cudaStream_t)stream);
}

size_t razer_gemm_mx_grouped_workspace_size(int64_t T, int64_t K, int64_t E) { return gemm_mx_online_workspace_bytes(T, K, E); }

}  // extern "C"
