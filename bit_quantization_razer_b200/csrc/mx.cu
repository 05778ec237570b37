// MXFP4 quantizer and decoder, and the rearrangement of row-major scale bytes
// into scale tiles.
//
// MXFP4 (OCP Microscaling Formats 1.0, 5.3 and 6.3): blocks of 32 E2M1
// elements along a row and one E8M0 scale per block.  With m the largest
// magnitude of a block,
//   e    = clamp(floor(log2 m) - 2, -127, 127)    (m = 0: -127; 2 = log2 of
//          E2M1's largest power of two, 4)
//   code = RN_E2M1(x * 2^-e), ties to the even code, magnitudes above 6 to 6
//   byte = e + 127; 255 (NaN), with codes of 0, for a block with a NaN or an
//          infinity.
// The scale is a power of two, so x * 2^-e is exact in binary32 (a product
// below its range rounds to code 0 either way) and the hardware E2M1 convert
// makes the only rounding.
#include "mx.cuh"

namespace razer {
namespace mx {

// eight 16-bit inputs in a 16-byte vector
template <typename T> struct Abs16;
template <> struct Abs16<__half> {
    static constexpr unsigned kInf = 0x7C00u;
    static __device__ __forceinline__ float to_f(unsigned b) { return __half2float(__ushort_as_half((unsigned short)b)); }
};
template <> struct Abs16<__nv_bfloat16> {
    static constexpr unsigned kInf = 0x7F80u;
    static __device__ __forceinline__ float to_f(unsigned b) { return __uint_as_float(b << 16); }
};

// four E2M1 codes pairs (8 nibbles, element 0 lowest) of 8 scaled values
__device__ __forceinline__ unsigned e2m1x8(const float (&v)[8])
{
    unsigned r;
    asm("{ .reg .b8 b0, b1, b2, b3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
        "mov.b32 %0, {b0, b1, b2, b3}; }"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// The scale byte of a block whose largest magnitude has the 16-bit pattern m,
// and 2^-e as a binary32
template <typename T> __device__ __forceinline__ unsigned scale_byte(unsigned m, float &inv)
{
    const unsigned field = __float_as_uint(Abs16<T>::to_f(m)) >> 23;  // binary32 exponent field
    const unsigned byte = m >= Abs16<T>::kInf ? 255u : (field > 2u ? field - 2u : 0u);
    inv = __uint_as_float((254u - (byte == 255u ? 0u : byte)) << 23);
    return byte;
}
__device__ __forceinline__ unsigned abs_max2(uint4 v)
{
    return __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
}
template <typename T> __device__ __forceinline__ unsigned encode8(uint4 v, float inv)
{
    const float2 a = In16<T>::to_f2(v.x), b = In16<T>::to_f2(v.y), c = In16<T>::to_f2(v.z), d = In16<T>::to_f2(v.w);
    const float s[8] = {a.x * inv, a.y * inv, b.x * inv, b.y * inv, c.x * inv, c.y * inv, d.x * inv, d.y * inv};
    return e2m1x8(s);
}

// A block of 32: its codes, and the scale byte as the result
template <typename T> __device__ __forceinline__ unsigned encode_block(const uint4 (&v)[4], uint4 &codes)
{
    const unsigned m2 = __vmaxu2(__vmaxu2(abs_max2(v[0]), abs_max2(v[1])), __vmaxu2(abs_max2(v[2]), abs_max2(v[3])));
    float inv;
    const unsigned byte = scale_byte<T>(max(m2 & 0xFFFFu, m2 >> 16), inv);
    codes = make_uint4(encode8<T>(v[0], inv), encode8<T>(v[1], inv), encode8<T>(v[2], inv), encode8<T>(v[3], inv));
    if (byte == 255u) codes = make_uint4(0u, 0u, 0u, 0u);
    return byte;
}

// a / b for a >= 0: the 64-bit division costs as much as encoding 16 values
__device__ __forceinline__ int64_t div_small(int64_t a, int64_t b) { return a <= UINT32_MAX ? (uint32_t)a / (uint32_t)b : a / b; }

// The offsets of up to kEdges - 1 groups in shared memory, where a search is
// cheap (through global memory it took half as long again as the quantizing);
// more stay where they are.
constexpr int kEdges = 256;
__device__ __forceinline__ const int32_t *stage_edges(const int32_t *offsets, int E, int32_t *edges)
{
    if (E == 0 || E >= kEdges) return offsets;
    for (int i = threadIdx.x; i <= E; i += blockDim.x) edges[i] = offsets[i];
    __syncthreads();
    return edges;
}

// Finds where the scales of a row start in their tile row; NULL: a row of no
// group, left as it is.  The warp looks up the group of its task's first row
// together, 32 offsets a step, and most lanes' rows lie in it; the others search
// for themselves (6000 x 4096 in 16 groups 12.6 us, every lane by itself 13.8;
// without groups, in a kernel that knows of none, 10.1, with the tests 10.6).
struct RowTiles {
    int row0, e, start, end;  // the first row, its group (start = end: none)
    __device__ __forceinline__ void find(int64_t first, int64_t M, const int32_t *offsets, int E)
    {
        row0 = (int)first;
        if (E == 0 || (row0 >= start && row0 < end)) return;
        const int lane = threadIdx.x & 31;
        int upto = 0;  // offsets that are at most row0
        for (int i = 0; i <= E; i += 32) {
            const unsigned some = __ballot_sync(0xffffffffu, i + lane <= E && group_edge(offsets, min(i + lane, E), (int)M) <= row0);
            upto += __popc(some);
            if (some != 0xffffffffu) break;
        }
        e = upto - 1;
        start = end = 0;
        if (e < 0 || e >= E) return;
        const int a = group_edge(offsets, e, (int)M), b = group_edge(offsets, e + 1, (int)M);
        if (a <= row0 && row0 < b) {  // offsets out of order may give a group that does not hold it
            start = a;
            end = b;
        }
    }
    __device__ __forceinline__ uint8_t *at(int64_t row, int64_t M, int64_t ct, const int32_t *offsets, int E, const uint8_t *tiles) const
    {
        int64_t trow = row / kTileRows;
        int in_tile = (int)(row % kTileRows);
        if (E > 0) {
            const int r = (int)row;
            int g = e, first = start;
            if (r < start || r >= end) {
                g = r == row0 ? -1 : group_of_row(offsets, E, (int)M, r);
                if (g < 0) return nullptr;
                first = group_edge(offsets, g, (int)M);
            }
            trow = group_tile_row(first, g) + (r - first) / kTileRows;
            in_tile = (r - first) % kTileRows;
        }
        return const_cast<uint8_t *>(tiles) + trow * ct * kTileBytes + (in_tile & 31) * 16 + (in_tile >> 5) * 4;
    }
};

// One lane per block of 32, 32 consecutive blocks of the matrix per warp and
// task: no shuffles for the largest magnitude, 16 bytes of codes a lane, half
// the instructions per element of four lanes that share a block.  The input
// comes through shared memory, where each warp has its next task in flight
// (cp.async, whole 512-byte lines) while it encodes one: registers for that
// would cost the occupancy it is meant to help.  16-byte piece j of lane l's
// block lies at piece 4 l + (j ^ (l / 2 % 4)), so that eight lanes' reads fall
// into different banks.
// Bound: HBM, 2 + 17/32 bytes an element.  14336 x 4096: 25.5 us, 5.8 TB/s
// (four lanes to a block and direct loads: 34 us).
constexpr int kQuantizeCtas = 4, kRing = 2;  // CTAs per SM: one wave

template <typename T, bool GROUPED>
__global__ void __launch_bounds__(256, kQuantizeCtas) quantize_mx_kernel(const T *__restrict__ x, int64_t M, int64_t K,
                                                                         const int32_t *offsets, int groups,
                                                                         uint8_t *__restrict__ codes, uint8_t *__restrict__ tiles)
{
    __shared__ uint4 ring[8][kRing][128];
    __shared__ int32_t edges[GROUPED ? kEdges : 1];
    const int E = GROUPED ? groups : 0;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    uint4(*mine)[128] = ring[threadIdx.x >> 5];
    const int64_t warp = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int64_t warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    const int64_t kb = K / 32, ct = tile_cols(false, K), nb = M * kb;
    if (E > 0 && blockIdx.x == 0 && threadIdx.x < 32) check_offsets(offsets, E, (int)M);
    offsets = stage_edges(offsets, E, edges);
    auto fetch = [&](int64_t task, int slot) {
        const uint4 *src = reinterpret_cast<const uint4 *>(x) + task * 128;
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const int i = lane + 32 * q, l = i >> 2, at = 4 * l + ((i ^ (l >> 1)) & 3);
            if (task * 32 + l < nb)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(&mine[slot][at])), "l"(src + i)
                             : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    RowTiles rt = {0, 0, 0, 0};
    int slot = 0;
#pragma unroll
    for (int i = 0; i < kRing - 1; i++) fetch(warp + i * warps, i);
    for (int64_t task = warp; task * 32 < nb; task += warps) {
        fetch(task + (kRing - 1) * warps, slot == 0 ? kRing - 1 : slot - 1);
        const int64_t blk = task * 32 + lane, row = div_small(blk, kb);
        if constexpr (GROUPED) rt.find(__shfl_sync(0xffffffffu, row, 0), M, offsets, E);
        const int c = (int)(blk - row * kb);
        uint8_t *t = blk < nb ? rt.at(row, M, ct, offsets, E, tiles) : nullptr;
        asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
        __syncwarp();
        uint4 v[4], out;
#pragma unroll
        for (int j = 0; j < 4; j++) v[j] = mine[slot][4 * lane + ((j ^ (lane >> 1)) & 3)];
        __syncwarp();  // read before the place is filled again
        slot = slot + 1 == kRing ? 0 : slot + 1;
        const unsigned byte = encode_block<T>(v, out);
        if (t) reinterpret_cast<uint4 *>(codes)[blk] = out;
        if ((kb & 3) == 0) {
            // four lanes hold the four scales of a word
            unsigned word = byte << (8 * (lane & 3));
            word |= __shfl_xor_sync(0xffffffffu, word, 1);
            word |= __shfl_xor_sync(0xffffffffu, word, 2);
            if ((lane & 3) == 0 && t) *reinterpret_cast<unsigned *>(t + (c >> 2) * kTileBytes) = word;
        } else if (t) {
            t += (c >> 2) * kTileBytes + (c & 3);
            *t = (uint8_t)byte;
            if (c + 1 == kb)  // the row's last word: zeros behind its scales
                for (int i = c + 1; i & 3; i++) *++t = 0;
        }
    }
}

// f16 pairs of 4 or 8 E2M1 codes
template <int PAIRS> __device__ __forceinline__ void e2m1_pairs(unsigned w, unsigned (&h)[PAIRS])
{
    if constexpr (PAIRS == 4)
        asm("{ .reg .b8 b0, b1, b2, b3; mov.b32 {b0, b1, b2, b3}, %4; "
            "cvt.rn.f16x2.e2m1x2 %0, b0; cvt.rn.f16x2.e2m1x2 %1, b1; cvt.rn.f16x2.e2m1x2 %2, b2; cvt.rn.f16x2.e2m1x2 %3, b3; }"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
            : "r"(w));
    else
        asm("{ .reg .b8 b0, b1; mov.b16 {b0, b1}, %2; "
            "cvt.rn.f16x2.e2m1x2 %0, b0; cvt.rn.f16x2.e2m1x2 %1, b1; }"
            : "=r"(h[0]), "=r"(h[1])
            : "h"((unsigned short)w));
}

// out = code * 2^(byte - 127), exact in binary32, rounded once to the output
// type.  A lane writes 16 bytes at a time, contiguous over the warp: 8 outputs
// of 16 bits or 4 of 32.
// 14336 x 4096 to fp32: 46 us, 5.8 TB/s of its 4.53 bytes an element (8 outputs
// a lane in two stores 32 bytes apart: 84 us).
constexpr int kTaskCols = 1024;  // columns of one row that a warp takes at a time

template <typename TOut>
__global__ void __launch_bounds__(256) dequant_mx_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ tiles, int64_t M,
                                                         int64_t K, int64_t chunks, const int32_t *offsets, int E,
                                                         TOut *__restrict__ out)
{
    __shared__ int32_t edges[kEdges];
    pdl_trigger();
    pdl_wait();
    constexpr int kPer = 16 / (int)sizeof(TOut), kIters = kTaskCols / (32 * kPer);
    const int lane = threadIdx.x & 31;
    const int64_t warp = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int64_t warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    const int64_t ct = tile_cols(false, K), total = M * chunks;
    if (E > 0 && blockIdx.x == 0 && threadIdx.x < 32) check_offsets(offsets, E, (int)M);
    offsets = stage_edges(offsets, E, edges);
    RowTiles rt = {0, 0, 0, 0};
    for (int64_t task = warp; task < total; task += warps) {
        const int64_t row = div_small(task, chunks);
        const int col = (int)(task - row * chunks) * kTaskCols;
        rt.find(row, M, offsets, E);
        const uint8_t *scales = rt.at(row, M, ct, offsets, E, tiles);
        if (!scales) continue;
        // one base pointer each, constant steps from it: with a 64-bit row * K + c
        // for every vector the kernel spent 79 instructions on four outputs
        const int left = (int)min((int64_t)kTaskCols, K - col) - kPer * lane;  // columns from this lane's first on
        const int64_t at = row * K + col + kPer * lane;
        const uint8_t *cp = codes + at / 2, *sp = scales + (int64_t)(col / 128) * kTileBytes;
        TOut *op = out + at;
        unsigned w[kIters], sb[kIters];
#pragma unroll
        for (int i = 0; i < kIters; i++) {
            constexpr int kCols = 32 * kPer;
            w[i] = sb[i] = 0u;
            if (kCols * i < left) {
                if constexpr (kPer == 8) w[i] = __ldg(reinterpret_cast<const unsigned *>(cp + kCols / 2 * i));
                else w[i] = __ldg(reinterpret_cast<const unsigned short *>(cp + kCols / 2 * i));
                const int c = kCols * i + kPer * lane;  // from a multiple of 128 on
                sb[i] = __ldg(sp + (c / 128) * kTileBytes + (c / 32) % 4);
            }
        }
#pragma unroll
        for (int i = 0; i < kIters; i++) {
            constexpr int kCols = 32 * kPer;
            if (kCols * i >= left) break;
            const float s = e8m0_value(sb[i]);
            unsigned h[kPer / 2];
            e2m1_pairs<kPer / 2>(w[i], h);
            float q[8];
#pragma unroll
            for (int j = 0; j < kPer / 2; j++) {
                const float2 p = In16<__half>::to_f2(h[j]);
                q[2 * j] = p.x * s;
                q[2 * j + 1] = p.y * s;
            }
            if constexpr (kPer == 4)
                *reinterpret_cast<float4 *>(op + kCols * i) = make_float4(q[0], q[1], q[2], q[3]);
            else
                *reinterpret_cast<uint4 *>(op + kCols * i) = make_uint4(Out16<TOut>::pack(q[0], q[1]), Out16<TOut>::pack(q[2], q[3]),
                                                                        Out16<TOut>::pack(q[4], q[5]), Out16<TOut>::pack(q[6], q[7]));
        }
    }
}

// Row-major scale bytes [R, C] -> tiles.  One CTA of 128 threads per tile row
// and 4 tiles: a thread reads 16 scales of its row, the tiles are put
// together in shared memory and leave it as whole 512-byte rows.  Rows and
// columns past the matrix become 0 (a scale of 0 or 2^-127: never a NaN that
// could meet the zero codes there).  Grouped: the rows of tile row t are
// those of the group that owns it; tile rows without rows stay as they are.
__global__ void __launch_bounds__(128) tile_scales_kernel(const uint8_t *__restrict__ rows, int64_t R, int64_t C, int64_t ct, int64_t col_chunks,
                                                          int64_t trows, const int32_t *__restrict__ offsets, int E, int vec,
                                                          uint8_t *__restrict__ tiles)
{
    __shared__ __align__(16) uint8_t buf[4 * kTileBytes];
    pdl_trigger();
    pdl_wait();
    const int64_t cc = blockIdx.x % col_chunks, tr = blockIdx.x / col_chunks;  // tr counts the tile rows of every batch
    const int i = threadIdx.x;
    int64_t row, end;
    if (E > 0 && blockIdx.x == 0 && threadIdx.x < 32) check_offsets(offsets, E, (int)R);
    if (E > 0) {
        // the last group whose first tile row is at most tr
        int lo = 0, hi = E;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (group_tile_row(group_edge(offsets, mid, (int)R), mid) <= tr) lo = mid;
            else hi = mid;
        }
        const int start = group_edge(offsets, lo, (int)R);
        const int64_t base = (int64_t)start + (tr - group_tile_row(start, lo)) * kTileRows;
        end = group_edge(offsets, lo + 1, (int)R);
        if (base < start || base >= end) return;  // no rows in this tile row (the same for the whole CTA)
        row = base + i;
    } else {
        const int64_t b = tr / trows;
        row = b * R + (tr - b * trows) * kTileRows + i;
        end = (b + 1) * R;
    }
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    const int64_t c0 = cc * 16;
    if (row < end) {
        const uint8_t *p = rows + row * C + c0;
        if (vec && c0 + 16 <= C) {
            v = *reinterpret_cast<const uint4 *>(p);
        } else {
            unsigned w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int j = 0; j < 16; j++)
                if (c0 + j < C) w[j >> 2] |= (unsigned)p[j] << (8 * (j & 3));
            v = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    const int at = (i & 31) * 16 + (i >> 5) * 4;
    *reinterpret_cast<unsigned *>(buf + at) = v.x;
    *reinterpret_cast<unsigned *>(buf + at + kTileBytes) = v.y;
    *reinterpret_cast<unsigned *>(buf + at + 2 * kTileBytes) = v.z;
    *reinterpret_cast<unsigned *>(buf + at + 3 * kTileBytes) = v.w;
    __syncthreads();
    const int64_t t = cc * 4 + (i >> 5);  // warp w writes tile w
    if (t < ct) reinterpret_cast<uint4 *>(tiles + (tr * ct + t) * kTileBytes)[i & 31] = reinterpret_cast<const uint4 *>(buf)[i];
}

// 8 warps a CTA, one wave of `per_sm` CTAs an SM at most
static unsigned mx_grid(int64_t warps_wanted, int per_sm)
{
    const int64_t g = (warps_wanted + 7) / 8, cap = (int64_t)sm_count() * per_sm;
    return (unsigned)(g < 1 ? 1 : (g > cap ? cap : g));
}

}  // namespace mx

razer_status run_quantize_mx(const void *X, razer_dtype dt, int64_t M, int64_t K, const int32_t *offsets, int E, uint8_t *codes,
                             uint8_t *tiles, cudaStream_t st)
{
    using namespace mx;
    const unsigned g = mx_grid((M * (K / 32) + 31) / 32, kQuantizeCtas);
    cudaError_t e;
    if (dt == RAZER_F16)
        e = launch_pdl(E > 0 ? quantize_mx_kernel<__half, true> : quantize_mx_kernel<__half, false>, g, 256u, 0, st,
                       reinterpret_cast<const __half *>(X), M, K, offsets, E, codes, tiles);
    else
        e = launch_pdl(E > 0 ? quantize_mx_kernel<__nv_bfloat16, true> : quantize_mx_kernel<__nv_bfloat16, false>, g, 256u, 0, st,
                       reinterpret_cast<const __nv_bfloat16 *>(X), M, K, offsets, E, codes, tiles);
    return e == cudaSuccess ? RAZER_OK : RAZER_ERR_CUDA;
}

razer_status run_dequant_mx(const uint8_t *codes, const uint8_t *tiles, int64_t M, int64_t K, const int32_t *offsets, int E, void *out,
                            razer_dtype dt, cudaStream_t st)
{
    using namespace mx;
    const int64_t chunks = (K + kTaskCols - 1) / kTaskCols;
    const unsigned g = mx_grid(M * chunks, 16);
    cudaError_t e;
    if (dt == RAZER_F32)
        e = launch_pdl(dequant_mx_kernel<float>, g, 256u, 0, st, codes, tiles, M, K, chunks, offsets, E, reinterpret_cast<float *>(out));
    else if (dt == RAZER_F16)
        e = launch_pdl(dequant_mx_kernel<__half>, g, 256u, 0, st, codes, tiles, M, K, chunks, offsets, E, reinterpret_cast<__half *>(out));
    else
        e = launch_pdl(dequant_mx_kernel<__nv_bfloat16>, g, 256u, 0, st, codes, tiles, M, K, chunks, offsets, E, reinterpret_cast<__nv_bfloat16 *>(out));
    return e == cudaSuccess ? RAZER_OK : RAZER_ERR_CUDA;
}

razer_status run_tile_scales(const uint8_t *rows, int64_t batch, int64_t R, int64_t C, const int32_t *offsets, int E, uint8_t *tiles,
                             cudaStream_t st)
{
    using namespace mx;
    const int64_t ct = (C + 3) / 4, col_chunks = (ct + 3) / 4;
    const int64_t trows = E > 0 ? tile_rows_grouped(R, E) : tile_rows(R);
    const int vec = (C % 16 == 0 && (reinterpret_cast<uintptr_t>(rows) & 15) == 0) ? 1 : 0;
    const cudaError_t e = launch_pdl(tile_scales_kernel, (unsigned)(batch * trows * col_chunks), 128u, 0, st, rows, R, C, ct, col_chunks, trows, offsets, E, vec, tiles);
    return e == cudaSuccess ? RAZER_OK : RAZER_ERR_CUDA;
}

}  // namespace razer
