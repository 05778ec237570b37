// Scale tiles and row groups of the microscaled 4-bit operators (MXFP4, and
// NVFP4 where its operands go to the tensor cores packed).
//
// Scale tiles: the block-scaled MMA reads its scale bytes from tensor memory,
// 128 rows x 4 scales at a time, and tcgen05.cp fills that from 512
// contiguous bytes of shared memory.  Packed tensors therefore keep their
// scale bytes in tiles of 128 rows x 4 scales, row-major over the tiles:
//   byte (r % 32) * 16 + (r % 128) / 32 * 4 + c % 4  of tile (r / 128, c / 4),
// so that a kernel moves whole tiles with bulk copies and rearranges nothing.
//
// Row groups: rows sorted by expert, group e = rows offsets[e] ..
// offsets[e + 1] - 1.  A group's scales start a tile row of their own,
//   tile row of row r = offsets[e] / 128 + e + (r - offsets[e]) / 128:
// floor((a + n) / 128) + 1 - floor(a / 128) >= ceil(n / 128), so the groups
// never overlap, T / 128 + E tile rows hold them all, and no prefix sum over
// the groups is needed.
#pragma once
#include "razer_internal.cuh"

namespace razer {
namespace mx {

constexpr int kTileRows = 128;
constexpr int kTileBytes = 512;

__host__ __device__ constexpr int block_of(bool nv) { return nv ? 16 : 32; }
// scale tiles along K of a row of K elements
__host__ __device__ constexpr int64_t tile_cols(bool nv, int64_t K) { return (K / block_of(nv) + 3) / 4; }
// tile rows of R rows, or of T rows in E groups
__host__ __device__ constexpr int64_t tile_rows(int64_t R) { return (R + kTileRows - 1) / kTileRows; }
__host__ __device__ constexpr int64_t tile_rows_grouped(int64_t T, int64_t E) { return T / kTileRows + E; }

// offsets[i] brought into 0..T: an array that breaks the rules (negative,
// beyond T) reads and writes inside the buffers all the same
__device__ __forceinline__ int group_edge(const int32_t *offsets, int i, int T)
{
    const int v = offsets[i];
    return v < 0 ? 0 : (v > T ? T : v);
}
// reports offsets that break the rules in the device status word (one warp of a launch calls it)
__device__ __forceinline__ void check_offsets(const int32_t *offsets, int E, int T)
{
    for (int i = threadIdx.x & 31; i <= E; i += 32) {
        const int v = __ldg(offsets + i);
        if (v < 0 || v > T || (i > 0 && v < __ldg(offsets + i - 1))) set_device_status(RAZER_ERR_INVALID_ARG);
    }
}
// first tile row of a group that starts at row `start`
__device__ __forceinline__ int group_tile_row(int start, int e) { return start / kTileRows + e; }

// the group whose rows hold r: the last e with offsets[e] <= r, or -1
__device__ __forceinline__ int group_of_row(const int32_t *offsets, int E, int T, int r)
{
    int lo = 0, hi = E;  // offsets[lo] <= r < offsets[hi]
    if (r < group_edge(offsets, 0, T) || r >= group_edge(offsets, E, T)) return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (group_edge(offsets, mid, T) <= r) lo = mid;
        else hi = mid;
    }
    return lo;
}

// 2^(b - 127) of an E8M0 byte (0: 2^-127, a binary32 subnormal; 255: NaN)
__device__ __forceinline__ float e8m0_value(unsigned b)
{
    return __uint_as_float(b == 0 ? 0x00400000u : (b == 255u ? 0x7FC00000u : b << 23));
}

}  // namespace mx
}  // namespace razer
