// Products of packed 4-bit operands on the block-scaled tcgen05 tensor cores
// (MXFP4 and NVFP4), dense or grouped by expert.
//
//   Y[m, n] = ts_a * ts_w * sum_k (q*s)_a[m, k] * (q*s)_w[n, k],   fp32 accumulation
//
// Both operands stay packed from HBM to the MMA (kind::mxf4nvf4: E2M1 x E2M1
// with the block scales applied inside the instruction), so nothing is
// decoded by the SM's lanes and a weight costs its 17/32 (MXFP4) or 9/16
// (NVFP4) bytes of traffic.
//
// The weights are the MMA's A operand (128 of their rows are the 128 lanes of
// the accumulator), the activation rows its B operand (the accumulator's
// columns): a call with few rows then uses a narrow MMA instead of a mostly
// empty 128-row tile, and a warp's store of one column writes 32 consecutive
// outputs of one row.
//
// Every wait is bounded (~2 s of globaltimer): on expiry the kernel records
// RAZER_ERR_TIMEOUT, the other roles stop at their next wait, copies in
// flight are waited for (bounded) and the tensor memory is freed.
#include "mx.cuh"
#include "sm100_async.cuh"

namespace razer {
namespace mx {

using gemm::smem_desc_k128;
using gemm::store1;
using gemm::tc_fence_after;
using gemm::tc_fence_before;
using gemm::tmem_ld32;
using gemm::umma_commit;

// Shared-memory descriptor of one scale tile for tcgen05.cp: 32 rows of 16
// bytes, no swizzle, 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr)
{
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}

// 512 bytes (128 rows x 4 scales) to 4 columns of tensor memory, the 32 lanes
// repeated for the four warps' quarters
__device__ __forceinline__ void scale_copy(uint32_t taddr, uint64_t desc)
{
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Instruction descriptor of kind::mxf4nvf4: E2M1 operands (type code 1), K =
// 64, scales E8M0 (1) or E4M3 (0); sf_id picks the first of the scale bytes
// this instruction uses out of each 4-byte word (2 of 4 bytes per 64 elements
// of MXFP4: 0 or 2; all 4 of NVFP4: 0).
__host__ __device__ constexpr uint32_t idesc_fp4(bool nv, int M, int N, int sf_id)
{
    return ((uint32_t)sf_id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((nv ? 0u : 1u) << 23) | ((uint32_t)(M >> 7) << 27) |
           ((uint32_t)sf_id << 29);
}

template <bool NV>
__device__ __forceinline__ void umma_fp4(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t acc)
{
    if constexpr (NV)
        asm volatile(
            "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%5], [%6], p; }" ::"r"(d),
            "l"(ad), "l"(bd), "r"(idesc), "r"(acc), "r"(sfa), "r"(sfb)
            : "memory");
    else
        asm volatile(
            "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p; }" ::"r"(d),
            "l"(ad), "l"(bd), "r"(idesc), "r"(acc), "r"(sfa), "r"(sfb)
            : "memory");
}

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// One product: N, K of the weights, T activation rows (in all groups), E = 0:
// dense.  tiles_w holds trows_w tile rows per expert, ct tiles each.
struct Problem {
    const uint8_t *tiles_a, *tiles_w;
    const float *ts_a, *ts_w;  // NULL: 1
    const int32_t *offsets;
    int E, T, N, K, ct, trows_w, gate;
};

// Where a unit of work lies: rows row0 .. row0 + count - 1 of the activations
// and the tile row where their scales start.
struct RowUnit {
    int e, row0, count, trow;
};

// The t-th piece of up to `step` rows (a multiple of 128, so that its scales
// start a tile row), counted over the groups; a warp works it out together,
// 32 groups at a time.  count = 0: there is no such piece.
__device__ __forceinline__ RowUnit row_unit(const Problem &p, int t, int step)
{
    RowUnit u = {0, 0, 0, 0};
    if (p.E == 0) {
        u.row0 = t * step;
        u.count = min(step, p.T - u.row0);
        u.trow = u.row0 / kTileRows;
        return u;
    }
    const int lane = threadIdx.x & 31;
    int before = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
        const int e = e0 + lane;
        int start = 0, n = 0;
        if (e < p.E) {
            start = group_edge(p.offsets, e, p.T);
            n = group_edge(p.offsets, e + 1, p.T) - start;
            if (n < 0) n = 0;
        }
        const int pieces = (n + step - 1) / step;
        int upto = pieces;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += o;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + upto > t);
        if (hit) {
            const int src = __ffs(hit) - 1;
            const int first = before + __shfl_sync(0xffffffffu, upto - pieces, src);
            start = __shfl_sync(0xffffffffu, start, src);
            n = __shfl_sync(0xffffffffu, n, src);
            const int in = (t - first) * step;
            u.e = e0 + src;
            u.row0 = start + in;
            u.count = min(step, n - in);
            u.trow = group_tile_row(start, u.e) + in / kTileRows;
            return u;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    return u;
}

// ---------------------------------------------------------------------------
// mx_stream_kernel: few rows per group.  One CTA per 128 weight rows x up to
// 128 activation rows: its time is the weights' way from HBM, so the ring of
// stages is what matters: two CTAs share an SM, and a stage holds only as many
// activation rows (in boxes of 32) as the unit has, so that few rows leave
// room for more stages (5 of 22 KB for up to 32 rows, 3 of 34 KB for 128).
//   warp 0: bulk-tensor producer; warp 1: tensor memory, MMA issuer;
//   warps 2-5: epilogue, one quarter of the accumulator's lanes each.
// Stage: 256 k of 128 weight rows (16 KB) and of the activation rows, and the
// scale tiles of both.
// ---------------------------------------------------------------------------
constexpr int kStepK = 256;  // a stage is 128 bytes of codes per row
template <bool NV> constexpr int kStepTiles = kStepK / (4 * (NV ? 16 : 32));  // scale tiles along a stage: 4 or 2
constexpr int kStreamThreads = 192;

constexpr int kStreamRows = 128, kBoxRows = 32;
// two CTAs per SM: 227 KB / 2 less 1 KB each that the system keeps
constexpr uint32_t kStreamRing = 115200u - 1024u - 512u, kStreamSmem = kStreamRing + 512u + 1024u;
constexpr int kStreamMaxStages = 8;

template <bool NV> struct StreamCfg {
    static constexpr uint32_t kA = 128 * 128, kBox = kBoxRows * 128, kS = kStepTiles<NV> * kTileBytes;
    // tensor memory: accumulator, then two sets of scales (A, B)
    static constexpr uint32_t kScaleCols = kStepTiles<NV> * 4;
    static constexpr uint32_t kCols = 256;
    static_assert(kStreamRows + 4 * kScaleCols <= kCols, "two CTAs share an SM's tensor memory");
    static_assert(kStreamRing / (kA + kBox + 2 * kS) <= kStreamMaxStages, "barriers for every stage");
    static_assert(kStreamRing / (kA + kStreamRows * 128 + 2 * kS) >= 3, "a ring for the widest unit");
};

template <bool NV, typename TOut>
__global__ void __launch_bounds__(kStreamThreads, 2)
    mx_stream_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ Problem p,
                     int ntiles, TOut *__restrict__ Y, int inject_stall)
{
    using Cfg = StreamCfg<NV>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *bars = smem + kStreamRing;
    const uint32_t full = smem_addr(bars), empty = full + 8 * kStreamMaxStages, acc_full = empty + 8 * kStreamMaxStages, drained = acc_full + 8;
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(bars + 256);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 260);
    volatile int *unit_slot = reinterpret_cast<volatile int *>(bars + 264);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n0 = (int)(blockIdx.x % (unsigned)ntiles) * 128, t = (int)(blockIdx.x / (unsigned)ntiles);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStreamMaxStages; s++) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(drained, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr((const void *)tmem_slot)),
                     "n"(Cfg::kCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    pdl_wait();  // the activations come from an earlier kernel of the stream
    if (p.E > 0 && blockIdx.x == 0) check_offsets(p.offsets, p.E, p.T);
    if (warp == 0) {
        const RowUnit u = row_unit(p, t, kStreamRows);
        if (lane == 0) {
            unit_slot[0] = u.e;
            unit_slot[1] = u.row0;
            unit_slot[2] = u.count;
            unit_slot[3] = u.trow;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int ue = unit_slot[0], row0 = unit_slot[1], count = unit_slot[2], trow = unit_slot[3];
    const int nk = count > 0 ? (p.K + kStepK - 1) / kStepK : 0;
    const int boxes = (count + kBoxRows - 1) / kBoxRows;
    const uint32_t bbytes = (uint32_t)boxes * Cfg::kBox, stage = Cfg::kA + bbytes + 2 * Cfg::kS;
    const uint32_t stages = kStreamRing / stage;

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- producer ----------------
            const uint8_t *sw = p.tiles_w + ((int64_t)ue * p.trows_w + n0 / kTileRows) * p.ct * kTileBytes;
            const uint8_t *sa = p.tiles_a + (int64_t)trow * p.ct * kTileBytes;
            const int wrow = ue * p.N + n0;
            int g = 0;
            uint32_t s = 0, ph = 0;  // the ring: stage, how often it went round
            bool ok = true;
            for (; g < nk; g++) {
                if (!mbar_wait(empty + 8 * s, ph ^ 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                // fault injection (tests only): the first CTA never fills its first stage
                const bool stall = inject_stall && blockIdx.x == 0 && g == 0;
                const uint32_t a0 = smem_addr(smem) + s * stage, f = full + 8 * s;
                const int c0 = g * kStepTiles<NV>;
                const uint32_t sbytes = (uint32_t)min(kStepTiles<NV>, p.ct - c0) * kTileBytes;
                if (!stall) {
                    mbar_expect_tx(f, Cfg::kA + bbytes + 2 * sbytes);
                    tma_load_2d(a0, &tmap_w, g * 128, wrow, f);
                    for (int b = 0; b < boxes; b++) tma_load_2d(a0 + Cfg::kA + b * Cfg::kBox, &tmap_a, g * 128, row0 + b * kBoxRows, f);
                    bulk_load(a0 + Cfg::kA + bbytes, sw + (int64_t)c0 * kTileBytes, sbytes, f);
                    bulk_load(a0 + Cfg::kA + bbytes + Cfg::kS, sa + (int64_t)c0 * kTileBytes, sbytes, f);
                }
                if (++s == stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (!ok) {
                // let the loads already issued land before the CTA exits (bounded)
                const uint64_t t0 = globaltimer();
                for (int gg = g > (int)stages ? g - (int)stages : 0; gg < g; gg++) {
                    if (inject_stall && blockIdx.x == 0 && gg == 0) continue;
                    while (!mbar_try_wait(full + 8 * ((uint32_t)gg % stages), ((uint32_t)gg / stages) & 1u) && globaltimer() - t0 < kTimeoutNs) {
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && nk > 0) {
            // ---------------- MMA issuer ----------------
            const int n = (count + 7) & ~7;  // the MMA's width: a multiple of 8
            const uint32_t id0 = idesc_fp4(NV, 128, n, 0), id2 = idesc_fp4(NV, 128, n, 2);
            uint32_t s = 0, ph = 0;
            bool ok = true;
            for (int g = 0; g < nk; g++) {
                if (!mbar_wait(full + 8 * s, ph, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t a0 = smem_addr(smem) + s * stage, b0 = a0 + Cfg::kA;
                const uint32_t sfa = tmem + kStreamRows + (uint32_t)(g & 1) * 2 * Cfg::kScaleCols, sfb = sfa + Cfg::kScaleCols;
                const int nt = min(kStepTiles<NV>, p.ct - g * kStepTiles<NV>);
                for (int i = 0; i < nt; i++) {
                    scale_copy(sfa + 4 * i, scale_desc(b0 + bbytes + i * kTileBytes));
                    scale_copy(sfb + 4 * i, scale_desc(b0 + bbytes + Cfg::kS + i * kTileBytes));
                }
                const int ks = min(4, (p.K - g * kStepK + 63) / 64);  // MMAs of 64 k that hold any of K
                for (int k = 0; k < ks; k++) {
                    const int word = NV ? k : k >> 1;
                    umma_fp4<NV>(tmem, smem_desc_k128(a0 + 32 * k), smem_desc_k128(b0 + 32 * k), (!NV && (k & 1)) ? id2 : id0, sfa + 4 * word,
                                 sfb + 4 * word, (g > 0 || k > 0) ? 1u : 0u);
                }
                umma_commit(empty + 8 * s);
                if (++s == stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (ok) umma_commit(acc_full);
            // every MMA issued has completed before the tensor memory is freed (bounded)
            umma_commit(drained);
            const uint64_t t0 = globaltimer();
            while (!mbar_try_wait(drained, 0) && globaltimer() - t0 < kTimeoutNs) {
            }
        }
    } else if (count > 0) {
        // ---------------- epilogue ----------------
        const int q = warp & 3;  // the quarter of the lanes this warp may read
        const int n = n0 + q * 32 + lane;
        float scale = 1.0f;
        if (p.ts_a) scale = __fmul_rn(scale, *p.ts_a);
        if (p.ts_w) scale = __fmul_rn(scale, p.ts_w[ue]);
        const int64_t ldy = p.gate ? p.N / 2 : p.N;
        if (mbar_wait_warp(acc_full, 0, abort_flag)) {
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < count; c0 += 32) {
                float v[32];
                tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)c0, v);
#pragma unroll
                for (int i = 0; i < 32; i++) {
                    float y = v[i] * scale;
                    if (p.gate) {
                        // row 2j gates row 2j + 1
                        const float up = __shfl_xor_sync(0xffffffffu, y, 1);
                        if (c0 + i < count && n < p.N && !(lane & 1)) store1<TOut>(Y + (int64_t)(row0 + c0 + i) * ldy + n / 2, silu_mul(y, up));
                    } else if (c0 + i < count && n < p.N) {
                        store1<TOut>(Y + (int64_t)(row0 + c0 + i) * ldy + n, y);
                    }
                }
            }
        }
        tc_fence_before();
    }
    __syncwarp();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(Cfg::kCols));
    }
}

// K = 0: empty sums.  Zero for the rows of the groups (dense: for every row).
template <typename TOut>
__global__ void __launch_bounds__(256) mx_zero_kernel(const int32_t *__restrict__ offsets, int E, int T, int64_t cols, TOut *__restrict__ Y)
{
    const int64_t lo = E > 0 ? group_edge(offsets, 0, T) : 0, hi = E > 0 ? group_edge(offsets, E, T) : T;
    for (int64_t i = lo * cols + (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < hi * cols; i += (int64_t)gridDim.x * blockDim.x)
        store1<TOut>(Y + i, 0.0f);
}

// a [rows, K / 2] byte matrix read in boxes of 128 bytes x box_rows, 128-byte swizzle
static bool encode_codes_map(CUtensorMap *map, const void *base, int64_t rows, int64_t K, int box_rows)
{
    const EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)(K / 2), (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(K / 2)};
    const cuuint32_t box[2] = {128u, (cuuint32_t)box_rows};
    const cuuint32_t es[2] = {1u, 1u};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// pieces of `step` rows that T rows in E groups can make
static int64_t max_pieces(int64_t T, int64_t E, int64_t step) { return E == 0 ? (T + step - 1) / step : T / step + (E < T ? E : T); }

template <bool NV, typename TOut>
static razer_status launch_stream(const uint8_t *codes_a, const uint8_t *codes_w, const Problem &p, TOut *Y, cudaStream_t st)
{
    static bool attr_set[64] = {false};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        if (cudaFuncSetAttribute(mx_stream_kernel<NV, TOut>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kStreamSmem) != cudaSuccess)
            return RAZER_ERR_CUDA;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    CUtensorMap mw, ma;
    if (!encode_codes_map(&mw, codes_w, (int64_t)p.N * (p.E ? p.E : 1), p.K, 128) || !encode_codes_map(&ma, codes_a, p.T, p.K, kBoxRows))
        return RAZER_ERR_CUDA;
    const int ntiles = (p.N + 127) / 128;
    const int64_t grid = max_pieces(p.T, p.E, kStreamRows) * ntiles;
    if (grid > INT32_MAX) return RAZER_ERR_SHAPE;
    const int inject = fault_injection_enabled() ? 1 : 0;
    if (launch_pdl(mx_stream_kernel<NV, TOut>, (unsigned)grid, (unsigned)kStreamThreads, (size_t)kStreamSmem, st, mw, ma, p, ntiles, Y,
                   inject) != cudaSuccess)
        return RAZER_ERR_CUDA;
    return RAZER_OK;
}

template <bool NV, typename TOut>
static razer_status launch_mx(const uint8_t *codes_a, const uint8_t *codes_w, const Problem &p, TOut *Y, cudaStream_t st)
{
    return launch_stream<NV, TOut>(codes_a, codes_w, p, Y, st);
}

template <typename TOut>
static razer_status run_mx_t(bool nv, const uint8_t *codes_a, const uint8_t *codes_w, const Problem &p, TOut *Y, cudaStream_t st)
{
    if (p.K == 0) {
        const int64_t cols = p.gate ? p.N / 2 : p.N;
        mx_zero_kernel<TOut><<<sm_count() * 4, 256, 0, st>>>(p.offsets, p.E, p.T, cols, Y);
        return last_launch_status();
    }
    return nv ? launch_mx<true, TOut>(codes_a, codes_w, p, Y, st) : launch_mx<false, TOut>(codes_a, codes_w, p, Y, st);
}

}  // namespace mx

// E = 0: dense (offsets ignored); otherwise W is [E, N, K] and ts_w holds E
// scales.  The caller has checked every argument; T, N > 0.
razer_status run_gemm_mx(const uint8_t *codes_a, const uint8_t *tiles_a, const float *ts_a, int64_t T, const int32_t *offsets, int E,
                         const uint8_t *codes_w, const uint8_t *tiles_w, const float *ts_w, razer_format fmt, int64_t N, int64_t K, int gate,
                         void *Y, razer_dtype out_dt, cudaStream_t st)
{
    const bool nv = fmt == RAZER_FMT_NVFP4;
    mx::Problem p;
    p.tiles_a = tiles_a;
    p.tiles_w = tiles_w;
    p.ts_a = ts_a;
    p.ts_w = ts_w;
    p.offsets = offsets;
    p.E = E;
    p.T = (int)T;
    p.N = (int)N;
    p.K = (int)K;
    p.ct = (int)mx::tile_cols(nv, K);
    p.trows_w = (int)mx::tile_rows(N);
    p.gate = gate;
    if (out_dt == RAZER_F32) return mx::run_mx_t<float>(nv, codes_a, codes_w, p, reinterpret_cast<float *>(Y), st);
    if (out_dt == RAZER_F16) return mx::run_mx_t<__half>(nv, codes_a, codes_w, p, reinterpret_cast<__half *>(Y), st);
    return mx::run_mx_t<__nv_bfloat16>(nv, codes_a, codes_w, p, reinterpret_cast<__nv_bfloat16 *>(Y), st);
}

}  // namespace razer
