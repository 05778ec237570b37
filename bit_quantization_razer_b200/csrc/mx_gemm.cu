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
// The allocation of tensor memory has no bound of its own: it waits until the
// other CTAs of the SM have left enough.  Whoever holds some must therefore be
// able to end without this CTA.  A programmatic dependent is not: it may have
// allocated, and then waits in griddepcontrol.wait for this grid.  So the one
// warp that allocates also lets the dependents in, and only once it has its
// columns; no other warp may (one thread's trigger counts for its CTA).
#include <algorithm>
#include <type_traits>

#include "mx.cuh"
#include "per_device.h"
#include "sm100_async.cuh"
#include "sm100_mma.cuh"

namespace razer {
namespace mx {

using gemm::store1;
using gemm::tc_fence_after;
using gemm::tc_fence_before;
using gemm::tmem_ld32;

// One lane of a converged warp, the same one every time.  The issuing loops
// below run in the whole warp and only the tcgen05 and copy instructions are
// left to this lane: loop control, addresses and descriptors are then uniform
// values.  With the whole loop inside `if (lane == 0)` every operand went
// through a per-thread register first, and a stage of 4 MMAs and 6 scale
// copies took 0.87 us (4096 x 4096 x 4096) where its MMAs need 0.2.
__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t e;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(e));
    return e;
}

// Whole-warp bounded wait whose result is uniform.
__device__ __forceinline__ bool mbar_wait_all(uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
}

// Whether the phase is over, without waiting: asked a stage ahead, so that the
// answer's latency (some 80 cycles) passes beside the instructions issued
// meanwhile.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}
// ... and the wait for it: `ready` is mbar_test's answer
__device__ __forceinline__ bool mbar_wait_tested(bool ready, uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    return __all_sync(0xffffffffu, ready) || mbar_wait_all(bar, parity, abort_flag);
}

// Shared-memory descriptors, the two 32-bit halves apart: codes (K-major,
// 128-byte swizzle, 8-row groups 1024 bytes apart) and one scale tile (32 rows
// of 16 bytes, no swizzle, 8-row groups 128 bytes apart).
constexpr uint32_t kCodesDescHi = (1024u >> 4) | (1u << 14) | (2u << 29), kScaleDescHi = (128u >> 4) | (1u << 14);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint64_t desc64(uint32_t hi, uint32_t lo) { return ((uint64_t)hi << 32) | lo; }

// 512 bytes (128 rows x 4 scales) to 4 columns of tensor memory, the 32 lanes
// repeated for the four warps' quarters (one lane issues)
template <bool PAIR>
__device__ __forceinline__ void scale_copy(uint32_t taddr, uint64_t desc)
{
    if constexpr (PAIR) asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    else asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Instruction descriptor of kind::mxf4nvf4: E2M1 operands (type code 1), K =
// 64, scales E8M0 (1) or E4M3 (0).  Scale ids 0 here: the ids (bits 4-5 and
// 29-30) pick the first of the scale bytes that the instruction takes of each
// 4-byte word (MXFP4 uses 2 per 64 elements, NVFP4 all 4).
__host__ __device__ constexpr uint32_t idesc_fp4(bool nv, int M, int N)
{
    return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((nv ? 0u : 1u) << 23) | ((uint32_t)(M >> 7) << 27);
}

#define RAZER_MX_MMA(GROUP, VEC)                                                                                                        \
    asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"                                                                               \
                 "tcgen05.mma.cta_group::" GROUP ".kind::mxf4nvf4.block_scale.scale_vec::" VEC " [%0], %1, %2, %3, [%5], [%6], p; }" ::"r"(d),  \
                 "l"(ad), "l"(bd), "r"(idesc), "r"(acc), "r"(sfa), "r"(sfb)                                                               \
                 : "memory")
template <bool NV, bool PAIR>
__device__ __forceinline__ void umma_fp4(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t acc)
{
    if constexpr (NV && PAIR) RAZER_MX_MMA("2", "4X");
    else if constexpr (NV) RAZER_MX_MMA("1", "4X");
    else if constexpr (PAIR) RAZER_MX_MMA("2", "2X");
    else RAZER_MX_MMA("1", "2X");
}
#undef RAZER_MX_MMA

// arrives on `bar` once the MMAs and copies issued so far are done (PAIR: on
// the barrier at this offset in both CTAs, `mask` of the cluster's ranks)
template <bool PAIR>
__device__ __forceinline__ void commit(uint32_t lead, uint32_t bar, uint16_t mask = 0)
{
    if constexpr (PAIR)
        asm volatile(
            "{ .reg .pred e; setp.ne.b32 e, %2, 0;\n"
            "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1; }" ::"r"(bar),
            "h"(mask), "r"(lead)
            : "memory");
    else
        asm volatile("{ .reg .pred e; setp.ne.b32 e, %1, 0;\n"
                     "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(bar),
                     "r"(lead)
                     : "memory");
}

constexpr int kStepK = 256;  // a stage is 128 bytes of codes per row
// stages of a row of K (K + kStepK may pass 2^31)
__host__ __device__ constexpr int stages_of(int K) { return K / kStepK + (K % kStepK != 0); }
template <bool NV> constexpr int kStepTiles = kStepK / (4 * (NV ? 16 : 32));  // scale tiles along a stage: 4 or 2

// The scale copies of one stage: kStepTiles tiles of the weights and of
// SFB_TILES tile rows of the activations.  A stage is always whole: the loads
// fill what lies past K with zero codes and zero scale bytes (0 or 2^-127,
// finite), which add nothing.
template <bool NV, bool PAIR, int SFB_TILES>
__device__ __forceinline__ void issue_scales(uint32_t lead, uint32_t sa0, uint32_t sb0, uint32_t sfa, uint32_t sfb)
{
    const uint32_t lsa = desc_lo(sa0), lsb = desc_lo(sb0);
    if (lead) {
#pragma unroll
        for (int i = 0; i < kStepTiles<NV>; i++) {
            scale_copy<PAIR>(sfa + 4 * i, desc64(kScaleDescHi, lsa + i * (kTileBytes >> 4)));
#pragma unroll
            for (int j = 0; j < SFB_TILES; j++)
                scale_copy<PAIR>(sfb + 4 * SFB_TILES * i + 4 * j, desc64(kScaleDescHi, lsb + (j * kStepTiles<NV> + i) * (kTileBytes >> 4)));
        }
    }
}

// The four MMAs of a stage, 64 k each; off2: the column of the activations'
// first scale tile that the unit starts at.
template <bool NV, bool PAIR, int SFB_TILES>
__device__ __forceinline__ void issue_mmas(uint32_t lead, uint32_t acc, uint32_t a0, uint32_t b0, uint32_t sfa, uint32_t sfb, uint32_t off2,
                                           uint32_t idesc, bool fresh)
{
    const uint32_t la = desc_lo(a0), lb = desc_lo(b0);
    if (lead) {
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const int word = NV ? k : k >> 1;
            // MXFP4: bytes 0-1 of a scale word, then 2-3 (scale ids 0 and 2)
            const uint32_t id = idesc | ((!NV && (k & 1)) ? (2u << 4) | (2u << 29) : 0u);
            umma_fp4<NV, PAIR>(acc, desc64(kCodesDescHi, la + 2 * k), desc64(kCodesDescHi, lb + 2 * k), id, sfa + 4 * word,
                               sfb + 4 * SFB_TILES * word + off2, (fresh && k == 0) ? 0u : 1u);
        }
    }
}

// silu(g) * u = g / (1 + exp(-g)) * u.  16-bit outputs take the hardware's
// 2^x and reciprocal.  Both flush what lies below binary32's normal range, so
// the quotient is formed as (g / 4) / (1/4 + exp(-g) / 4): the reciprocal then
// stays normal as long as exp(-g) is finite (g > -88.7), and below that is 0, as
// g / (1 + expf(-g)) is.  (With 1 / (1 + exp(-g)) as it stands, gates between
// -88.7 and -87.3 gave 0.)  The quarter of g comes with the scale that the sum
// is multiplied by anyway, kGate in the lanes that hold gates: another multiply
// here cost 1% (512 x 28672 x 4096 gated 31.8 -> 32.1 us).  Relative error: the
// exponent -g log2(e), at most 128, is off by 2^-18 of its own rounding and 128 *
// 2^-26 of the constant's, together 4e-6 of the power; the two functions add
// 2^-22 each: 5e-6, against the 2^-9 (2^-12) of the output's own rounding.  With
// expf and an IEEE division the epilogue of 512 x 28672 x 4096 took longer than
// its MMAs.
template <typename TOut> constexpr float kGate = sizeof(TOut) == 2 ? 0.25f : 1.0f;
// g is the gate times kGate
template <typename TOut> __device__ __forceinline__ float silu_mul(float g, float u)
{
    if constexpr (sizeof(TOut) == 2) {
        float e, r;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * (4.0f * -1.44269504f)));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(e, 0.25f, 0.25f)));
        return g * r * u;
    } else {
        return g / (1.0f + expf(-g)) * u;
    }
}

// One product: N, K of the weights, T activation rows (in all groups), E = 0:
// dense.  tiles_w holds trows_w tile rows per expert, ct tiles each.  pieces:
// how many the rows can make of those that the kernel takes at a time.
struct Problem {
    const uint8_t *tiles_a, *tiles_w;
    const float *ts_a, *ts_w;  // NULL: 1
    const int32_t *offsets;
    int E, T, N, K, ct, trows_w, gate, pieces;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

// Where a unit of work lies: rows row0 .. row0 + count - 1 of the activations
// and the tile row, and the row in it, where their scales start.
struct RowUnit {
    int e, row0, count, trow, off;
};

// Finds the t-th piece of up to `step` rows (a multiple of 64), counted over
// the groups, for a t that never falls: a warp keeps 32 groups at a time, a
// lane one of them, and loads the next 32 when t has passed these.  (Reading
// the offsets again for every unit cost each role some 0.4 us a unit.)
// No piece from p.pieces on is taken: whatever the offsets hold, a call has no
// more units than the host planned, and their numbers stay below 2^31.  (Offsets
// that alternate between 0 and T make E / 2 groups of T rows.)
struct RowWalk {
    int e0, before, start, n, upto, total;  // first group; pieces before it; this lane's group; its pieces' inclusive sum; all 32's

    // ceil(n / step); n + step may pass 2^31
    static __device__ __forceinline__ int pieces_of(int n, int step) { return n / step + (n % step != 0); }
    __device__ __forceinline__ void load(const Problem &p, int step)
    {
        const int lane = threadIdx.x & 31, e = e0 + lane;
        start = n = 0;
        if (e < p.E) {
            start = group_edge(p.offsets, e, p.T);
            n = max(group_edge(p.offsets, e + 1, p.T) - start, 0);
        }
        upto = pieces_of(n, step);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += o;
        }
        total = __shfl_sync(0xffffffffu, upto, 31);
    }
    __device__ __forceinline__ void begin(const Problem &p, int step)
    {
        e0 = before = 0;
        if (p.E > 0) load(p, step);
    }
    // count <= 0: there is no such piece
    __device__ __forceinline__ RowUnit at(const Problem &p, int t, int step)
    {
        RowUnit u = {0, 0, 0, 0, 0};
        if (t >= p.pieces) return u;
        if (p.E == 0) {
            u.row0 = t * step;
            u.count = min(step, p.T - u.row0);
            u.trow = u.row0 / kTileRows;
            u.off = u.row0 % kTileRows;
            return u;
        }
        while (t >= before + total) {
            if (e0 + 32 >= p.E) return u;
            before += total;
            e0 += 32;
            load(p, step);
        }
        const int src = __ffs(__ballot_sync(0xffffffffu, before + upto > t)) - 1;
        const int s0 = __shfl_sync(0xffffffffu, start, src), sn = __shfl_sync(0xffffffffu, n, src);
        const int last = before + __shfl_sync(0xffffffffu, upto, src), in = (t - last + pieces_of(sn, step)) * step;
        u.e = e0 + src;
        u.row0 = s0 + in;
        u.count = min(step, sn - in);
        u.trow = group_tile_row(s0, u.e) + in / kTileRows;
        u.off = in % kTileRows;
        return u;
    }
};

// a * scale and b * scale rounded to a word of 16-bit outputs, a in the low half
template <typename TOut> __device__ __forceinline__ unsigned pack_scaled(float a, float b, float scale)
{
    float x, y;
    asm("{ .reg .b64 p, s; mov.b64 p, {%2, %3}; mov.b64 s, {%4, %4}; mul.rn.f32x2 p, p, s; mov.b64 {%0, %1}, p; }"
        : "=f"(x), "=f"(y)
        : "f"(a), "f"(b), "f"(scale));
    return Out16<TOut>::pack(x, y);
}

// two adjacent 16-bit outputs (4-byte aligned)
template <typename TOut> __device__ __forceinline__ void store_pair(TOut *p, float a, float b)
{
    if constexpr (sizeof(TOut) == 2) *reinterpret_cast<unsigned *>(p) = Out16<TOut>::pack(a, b);
}

// Writes 32 columns of an accumulator: lane `lane` holds output column n of
// the rows row .. row + count - 1 (at most 32).  Adjacent lanes swap halves of
// two columns, so that the even lane finishes the first row and the odd lane
// the second: a gated pair meets in one lane and every lane computes one, and
// 16-bit outputs leave in pairs, 16 stores instead of 32; gated ones swap once
// more between lanes two apart, 8 stores.  Outputs without a gate are rounded
// first, so that one shuffle swaps both rows (4096 x 14336 x 512: 38.4 -> 33.5
// us).  ALL: 32 rows; the chains are then
// free of branches and run into each other (with a test between them a unit of
// 192 rows took 7,000 cycles, longer than its 16 stages of MMAs; with one store
// per column and lane and the gate tested inside the loop 15,700; now 3,100,
// gated 3,700).  Through shared memory, to leave it as whole lines: 46 us in
// place of 33.5, two barriers for every 8 rows.  PAIRS: rows of an even length, so that pairs are 4-byte
// aligned.
template <typename TOut, bool GATE, bool ALL, bool PAIRS>
__device__ __forceinline__ void write_columns_n(const float (&v)[32], float scale, TOut *__restrict__ Y, int64_t ldy, int count, bool mine, int n,
                                                int lane)
{
    const int odd = lane & 1, high = (lane >> 1) & 1;
    if (GATE && !odd) scale *= kGate<TOut>;  // this lane's sums are gates
    if constexpr (sizeof(TOut) == 2 && GATE && PAIRS) {
        // four rows a step; outputs n / 2 & ~1 and n / 2 | 1
        TOut *y = Y + (odd + 2 * high) * ldy + (n / 2 & ~1);
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            if (!ALL && i >= count) break;
            float r[2];
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const float keep = (odd ? v[i + 2 * j + 1] : v[i + 2 * j]) * scale, give = (odd ? v[i + 2 * j] : v[i + 2 * j + 1]) * scale;
                const float got = __shfl_xor_sync(0xffffffffu, give, 1);
                r[j] = silu_mul<TOut>(odd ? got : keep, odd ? keep : got);  // row 2j of the weights gates row 2j + 1
            }
            const float got = __shfl_xor_sync(0xffffffffu, high ? r[0] : r[1], 2);
            if (mine && (ALL || i + odd + 2 * high < count)) store_pair<TOut>(y, high ? got : r[0], high ? r[1] : got);
            y += 4 * ldy;
        }
    } else if constexpr (sizeof(TOut) == 2 && PAIRS) {
        // two rows a step, rounded before they are swapped: one shuffle for both
        TOut *y = Y + odd * ldy + (n & ~1);
        const unsigned halves = odd ? 0x3276u : 0x5410u;
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            if (!ALL && i >= count) break;
            const unsigned keep = pack_scaled<TOut>(v[i], v[i + 1], scale), got = __shfl_xor_sync(0xffffffffu, keep, 1);
            if (mine && (ALL || i + odd < count)) *reinterpret_cast<unsigned *>(y) = __byte_perm(keep, got, halves);
            y += 2 * ldy;
        }
    } else if constexpr (GATE) {
        // two rows a step
        TOut *y = Y + odd * ldy + n / 2;
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            if (!ALL && i >= count) break;
            const float keep = (odd ? v[i + 1] : v[i]) * scale, give = (odd ? v[i] : v[i + 1]) * scale;
            const float got = __shfl_xor_sync(0xffffffffu, give, 1);
            if (mine && (ALL || i + odd < count)) store1<TOut>(y, silu_mul<TOut>(odd ? got : keep, odd ? keep : got));
            y += 2 * ldy;
        }
    } else {
        TOut *y = Y + n;
#pragma unroll
        for (int i = 0; i < 32; i++) {
            if (!ALL && i >= count) break;
            if (mine) store1<TOut>(y, v[i] * scale);
            y += ldy;
        }
    }
}
template <typename TOut, bool GATE>
__device__ __forceinline__ void write_columns(const float (&v)[32], float scale, int N, TOut *__restrict__ Y, int64_t ldy, int row, int count,
                                              int n, int lane)
{
    const bool mine = n < N;
    TOut *y = Y + (int64_t)row * ldy;
    if (sizeof(TOut) == 2 && (ldy & 1) == 0) {
        if (count >= 32) write_columns_n<TOut, GATE, true, true>(v, scale, y, ldy, count, mine, n, lane);
        else write_columns_n<TOut, GATE, false, true>(v, scale, y, ldy, count, mine, n, lane);
    } else {
        if (count >= 32) write_columns_n<TOut, GATE, true, false>(v, scale, y, ldy, count, mine, n, lane);
        else write_columns_n<TOut, GATE, false, false>(v, scale, y, ldy, count, mine, n, lane);
    }
}

// shared-memory address of the same object in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Adds the sums that the CTAs of a cluster left in their shared memory (column c
// of lane r at (c * 128 + r) floats from `part`; CTA y of the split is rank
// rank0 + y * rank_step) and writes the outputs: columns in fours, dealt out
// over `workers` warps for each quarter of the lanes, added in the CTAs' order.
// One column at a time took 6 us for 64 columns over two CTAs, a remote load's
// latency each.
template <typename TOut, bool GATE>
__device__ __forceinline__ void join_sums(uint32_t part, int count, int splits, int rank0, int rank_step, int worker, int workers, int q, int n0,
                                          int N, TOut *__restrict__ Y, int row0, int lane)
{
    const int r = q * 32 + lane, n = n0 + r;
    const int64_t ldy = GATE ? N / 2 : N;
    for (int c = 4 * worker; c < count; c += 4 * workers) {
        float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int y = 0; y < splits; y++) {
            const uint32_t at = cluster_addr(part + (uint32_t)(c * 128 + r) * 4u, (uint32_t)(rank0 + y * rank_step));
#pragma unroll
            for (int j = 0; j < 4; j++) a[j] += ld_cluster(at + j * 512);  // past the last column: not written
        }
#pragma unroll
        for (int j = 0; j < 4; j++) {
            if constexpr (GATE) a[j] = silu_mul<TOut>(a[j] * kGate<TOut>, __shfl_xor_sync(0xffffffffu, a[j], 1));
            if (c + j < count && n < N && !(GATE && (lane & 1))) store1<TOut>(Y + (int64_t)(row0 + c + j) * ldy + (GATE ? n / 2 : n), a[j]);
        }
    }
}

// ---------------------------------------------------------------------------
// mx_stream_kernel: few rows per group.  A unit is 128 weight rows x up to 64
// activation rows; its time is the weights' way from HBM, so what matters is
// that copies never stop: two CTAs per SM, each a ring of stages that its
// producer fills across the units the CTA takes in turn, while two
// accumulators let the epilogue of one unit run beside the MMAs of the next.
//   warp 0: bulk-tensor producer; warp 1: tensor memory, MMA issuer;
//   warps 2-9: with TIn = void the epilogue alone, two warps per quarter of the
//   accumulator's lanes; otherwise they also quantize the activations (TIn
//   [T, K]) to MXFP4, stage by stage, straight into the shared-memory operand
//   and its scale tiles: a call with few rows is then one launch, reads X from
//   L2 and needs no workspace.
// Stage: 256 k of 128 weight rows (16 KB) and of `boxes` x 32 activation rows,
// and the scale tiles of both: 5 stages of 22 KB, or 4 of 26 KB.
// Where the units do not fill the SMs, the CTAs of a cluster share one: CTA z
// takes part z of K, leaves its fp32 sums in its own shared memory, and after
// a cluster barrier each CTA adds a share of the columns over the CTAs in
// order (deterministic; no workspace, no second launch).
// ---------------------------------------------------------------------------
constexpr int kStreamWorkers = 8, kStreamThreads = 64 + 32 * kStreamWorkers;
constexpr int kStreamRows = 64, kBoxRows = 32, kFuseRows = 16, kFuseGroupRows = 4;
// two CTAs per SM: 227 KB / 2 less 1 KB each that the system keeps
constexpr uint32_t kStreamRing = 115200u - 1024u - 512u, kStreamSmem = kStreamRing + 512u + 1024u;
constexpr int kStreamMaxStages = 8;

template <bool NV> struct StreamCfg {
    static constexpr uint32_t kA = 128 * 128, kBox = kBoxRows * 128, kS = kStepTiles<NV> * kTileBytes;
    // tensor memory: two accumulators, then the scales of a stage (weights, activations)
    static constexpr uint32_t kScaleCols = kStepTiles<NV> * 4;
    static constexpr uint32_t kCols = 256;
    static_assert(2 * kStreamRows + 2 * kScaleCols <= kCols, "two CTAs share an SM's tensor memory");
    static_assert(kStreamRing / (kA + kBox + 2 * kS) <= kStreamMaxStages, "barriers for every stage");
    static_assert(kStreamRing / (kA + kStreamRows * 128 + 2 * kS) >= 3, "a ring for the widest unit");
};
static_assert((kStreamRows + 3) * 128 * 4 <= kStreamRing, "the sums of a cluster's CTA");
// kFuseRows: up to so many rows a group, on average, an online call quantizes
// in the product.  Two launches / one, us: 14336 x 4096, 8 rows 10.7 / 9.2, 16
// rows 10.9 / 10.8, 24 rows 11.2 / 14.2; 28672 x 8192 24.8 / 24.2, 25.0 / 24.8,
// 25.2 / 33.3: every CTA quantizes all of its rows again.  kFuseGroupRows: the
// same for row groups, whose longest decides.  Random groups, two launches /
// one: 32 of 2048 x 4096, 4 rows 28.6 / 28.8, 8 rows 30.2 / 38.7; 43 of 466 x
// 13344, 4 rows 53.7 / 45.1, 8 rows 72 / 114; 64 of 512 x 2048, 6 rows 11.4 /
// 11.1, 16 rows 12.4 / 15.9.

template <bool NV, typename TOut, bool GATE, typename TIn>
__global__ void __launch_bounds__(kStreamThreads, 2)
    mx_stream_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_a,
                     const __grid_constant__ CUtensorMap tmap_sw, const __grid_constant__ CUtensorMap tmap_sa, const __grid_constant__ Problem p,
                     const TIn *__restrict__ X, int ntiles, int splits, int boxes, TOut *__restrict__ Y, int inject_stall)
{
    using Cfg = StreamCfg<NV>;
    constexpr bool kFused = !std::is_void<TIn>::value;
    static_assert(!(kFused && NV), "the quantizer writes MXFP4");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *bars = smem + kStreamRing;
    const uint32_t full = smem_addr(bars), empty = full + 8 * kStreamMaxStages, acc_full = empty + 8 * kStreamMaxStages, acc_empty = acc_full + 16,
                   drained = acc_empty + 16;
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(bars + 256);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 260);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int z = splits > 1 ? (int)cluster_rank() : 0, block = blockIdx.x / (unsigned)splits, blocks = gridDim.x / (unsigned)splits;
    const int steps = stages_of(p.K);
    // this CTA's stages of a unit: g0 .. g0 + nk - 1
    const int g0 = (int)((int64_t)steps * z / splits), nk = (int)((int64_t)steps * (z + 1) / splits) - g0;
    const uint32_t bbytes = (uint32_t)boxes * Cfg::kBox, stage = Cfg::kA + bbytes + 2 * Cfg::kS, stages = kStreamRing / stage;

    if (warp == 0) {
        // ---------------- producer ----------------
        // It sets up the barriers itself and does not wait for the other warps:
        // the first copies are on their way while they start.
        const uint32_t lead = elect_one();
        if (lead) {
            for (int s = 0; s < kStreamMaxStages; s++) {
                mbar_init(full + 8 * s, kFused ? 5 : 1);  // the producer, and the four warps that quantize the stage
                mbar_init(empty + 8 * s, 1);
            }
            for (int b = 0; b < 2; b++) {
                mbar_init(acc_full + 8 * b, 1);
                mbar_init(acc_empty + 8 * b, kStreamWorkers);
            }
            mbar_init(drained, 1);
            *abort_flag = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncwarp();
        asm volatile("barrier.cta.arrive 1, %0;" ::"n"(kStreamThreads) : "memory");
        pdl_wait();  // the operands may come from an earlier kernel of the stream
        uint32_t s = 0, ph = 0;  // the ring: stage, how often it went round
        bool ok = true, first = true;
        RowWalk walk;
        walk.begin(p, kStreamRows);
        for (int u = block; ok; u += blocks) {
            const RowUnit w = walk.at(p, u / ntiles, kStreamRows);
            if (w.count <= 0) break;
            const int n0 = u % ntiles * 128, wrow = w.e * p.N + n0, srow = w.e * p.trows_w + n0 / kTileRows;
            for (int g = 0; g < nk; g++) {
                if (!mbar_wait_all(empty + 8 * s, ph ^ 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                // fault injection (tests only): the first CTA never fills its first stage
                const bool stall = inject_stall && blockIdx.x == 0 && first;
                first = false;
                const uint32_t a0 = smem_addr(smem) + s * stage, f = full + 8 * s, s0 = a0 + Cfg::kA + bbytes;
                const int c0 = (g0 + g) * 128, t0 = (g0 + g) * kStepTiles<NV> * 2;
                if (lead && !stall) {
                    mbar_expect_tx(f, kFused ? Cfg::kA + Cfg::kS : stage);
                    tma_load_2d(a0, &tmap_w, c0, wrow, f);
                    tma_load_3d(s0, &tmap_sw, 0, t0, srow, f);
                    if constexpr (!kFused) {
                        // (a box without rows starts behind the unit's last: row0 + kBoxRows may pass 2^31)
                        for (int b = 0; b < boxes; b++)
                            tma_load_2d(a0 + Cfg::kA + b * Cfg::kBox, &tmap_a, c0, w.row0 + min(b * kBoxRows, w.count), f);
                        tma_load_3d(s0 + Cfg::kS, &tmap_sa, 0, t0, w.trow, f);
                    }
                }
                if (++s == stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (!ok) {
            // loads already issued land within microseconds; their barriers may
            // never complete: wait a fixed 2 ms before the CTA exits
            const uint64_t t0 = globaltimer();
            while (globaltimer() - t0 < 2000000ull) {
            }
            __syncwarp();
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr((const void *)tmem_slot)),
                     "n"(Cfg::kCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        pdl_trigger();  // not before: see the allocation's rule in the header of this file
        tc_fence_before();
        asm volatile("barrier.cta.sync 1, %0;" ::"n"(kStreamThreads) : "memory");
        tc_fence_after();
        pdl_wait();
        const uint32_t lead = elect_one(), tmem = *tmem_slot, sfa = tmem + 2 * kStreamRows, sfb = sfa + Cfg::kScaleCols;
        uint32_t s = 0, ph = 0, ti = 0;
        bool ok = true;
        RowWalk walk;
        walk.begin(p, kStreamRows);
        for (int u = block; ok; u += blocks, ti++) {
            const RowUnit w = walk.at(p, u / ntiles, kStreamRows);
            if (w.count <= 0) break;
            const uint32_t b = ti & 1u, acc = tmem + b * kStreamRows;
            // the epilogue has drained this accumulator
            if (!mbar_wait_all(acc_empty + 8 * b, ((ti >> 1) & 1u) ^ 1u, abort_flag)) break;
            const uint32_t idesc = idesc_fp4(NV, 128, (w.count + 7) & ~7);  // the MMA's width: a multiple of 8
            const uint32_t off2 = kFused ? 0u : (uint32_t)w.off >> 5;
            for (int g = 0; g < nk; g++) {
                if (!mbar_wait_all(full + 8 * s, ph, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t a0 = smem_addr(smem) + s * stage, b0 = a0 + Cfg::kA, s0 = b0 + bbytes;
                issue_scales<NV, false, 1>(lead, s0, s0 + Cfg::kS, sfa, sfb);
                issue_mmas<NV, false, 1>(lead, acc, a0, b0, sfa, sfb, off2, idesc, g == 0);
                commit<false>(lead, empty + 8 * s);
                if (++s == stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (ok) commit<false>(lead, acc_full + 8 * b);
        }
        // every MMA issued has completed before the tensor memory is freed (bounded)
        commit<false>(lead, drained);
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(drained, 0) && globaltimer() - t0 < kTimeoutNs) {
        }
        __syncwarp();
    } else {
        asm volatile("barrier.cta.sync 1, %0;" ::"n"(kStreamThreads) : "memory");
        tc_fence_after();
        pdl_wait();
        if (p.E > 0 && blockIdx.x == 0 && warp == 2) check_offsets(p.offsets, p.E, p.T);
        const uint32_t tmem = *tmem_slot;
        // ---------------- quantizer (of the unit with this CTA's number ti) ----------------
        // Warps 2-5 take the even stages, 6-9 the odd ones, a thread one block of
        // 32 at a time (16 rows are one block each); the block of the next stage
        // is on its way while this one is encoded.  (Two stages in turn: a warp
        // that took every fourth could be two rounds of the ring ahead, which a
        // barrier's parity cannot tell from none.)
        auto quantize = [&](const RowUnit &w, uint32_t ti) -> bool {
            if constexpr (kFused) {
                const int group = (warp - 2) >> 2, tid = (threadIdx.x - 64) & 127;
                uint4 v[4];
                auto load = [&](int g, int i) {
                    const int r = i >> 3;
                    const int64_t k = (int64_t)(g0 + g) * kStepK + 32 * (i & 7);
                    const bool in = g < nk && i < w.count * 8 && k < p.K;  // past K: zeros
                    const uint4 *x = reinterpret_cast<const uint4 *>(X + (int64_t)(w.row0 + r) * p.K + k);
#pragma unroll
                    for (int j = 0; j < 4; j++) v[j] = in ? __ldg(x + j) : make_uint4(0u, 0u, 0u, 0u);
                };
                const uint32_t base = ti * (uint32_t)nk;  // stages before this unit
                int g = (int)((base + (uint32_t)group) & 1u);
                load(g, tid);
                for (; g < nk; g += 2) {
                    const uint32_t s = (base + (uint32_t)g) % stages, ph = ((base + (uint32_t)g) / stages) & 1u;
                    if (!mbar_wait_all(empty + 8 * s, ph ^ 1u, abort_flag)) return false;
                    uint8_t *b0 = smem + s * stage + Cfg::kA, *sb = b0 + bbytes + Cfg::kS;
                    // 8 blocks a row: a block's 16 bytes of codes are one unit of the swizzle
                    for (int i = tid; i < w.count * 8; i += 128) {
                        const int r = i >> 3, c = i & 7;
                        uint4 codes;
                        const unsigned byte = encode_block<TIn>(v, codes);
                        load(i + 128 < w.count * 8 ? g : g + 2, i + 128 < w.count * 8 ? i + 128 : tid);
                        *reinterpret_cast<uint4 *>(b0 + r * 128 + ((c ^ (r & 7)) << 4)) = codes;
                        sb[(c >> 2) * kTileBytes + (r & 31) * 16 + (r >> 5) * 4 + (c & 3)] = (uint8_t)byte;
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full + 8 * s);
                }
            }
            return true;
        };
        // ---------------- epilogue ----------------
        const int q = warp & 3, c_first = ((warp - 2) >> 2) * 32, r = q * 32 + lane;  // quarter of the lanes; which of the columns
        const int64_t ldy = GATE ? p.N / 2 : p.N;
        const float ts_a = p.ts_a ? *p.ts_a : 1.0f;
        uint32_t ti = 0;
        RowWalk walk;
        walk.begin(p, kStreamRows);
        RowUnit w = walk.at(p, block / ntiles, kStreamRows);
        bool ok = w.count <= 0 || quantize(w, 0);
        for (int u = block; ok && w.count > 0; u += blocks, ti++) {
            // the next unit's stages are quantized before this one's sums are written:
            // its MMAs need them, and only its successor's this accumulator
            const RowUnit next = walk.at(p, (u + blocks) / ntiles, kStreamRows);
            if (next.count > 0 && !quantize(next, ti + 1)) break;
            const uint32_t b = ti & 1u;
            if (!mbar_wait_warp(acc_full + 8 * b, (ti >> 1) & 1u, abort_flag)) break;
            tc_fence_after();
            const int n = u % ntiles * 128 + r;
            const float scale = p.ts_w ? __fmul_rn(ts_a, p.ts_w[w.e]) : ts_a;
            float v[32];
            if (c_first < w.count) tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + b * kStreamRows + (uint32_t)c_first, v);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty + 8 * b);  // this warp has read its part: the accumulator goes back
            if (c_first < w.count) {
                if (splits == 1) {
                    write_columns<TOut, GATE>(v, scale, p.N, Y, ldy, w.row0 + c_first, w.count - c_first, n, lane);
                } else {
                    // the ring is free: the CTA's only unit has been read by its MMAs
                    float *part = reinterpret_cast<float *>(smem) + c_first * 128 + r;
#pragma unroll
                    for (int i = 0; i < 32; i++)
                        if (c_first + i < w.count) part[i * 128] = v[i] * scale;
                }
            }
            w = next;
        }
        tc_fence_before();
    }
    __syncwarp();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(*tmem_slot), "n"(Cfg::kCols));
    }
    if (splits > 1) {
        cluster_sync();  // every CTA's sums are written
        if (warp >= 2) {
            RowWalk walk;
            walk.begin(p, kStreamRows);
            const RowUnit w = walk.at(p, block / ntiles, kStreamRows);
            const int v = warp - 2;
            join_sums<TOut, GATE>(smem_addr(smem), w.count, splits, 0, 1, 2 * z + (v >> 2), 2 * splits, v & 3, block % ntiles * 128, p.N, Y, w.row0,
                                  lane);
        }
        __syncwarp();
        cluster_sync();  // no CTA leaves while another reads its sums
    }
}

// ---------------------------------------------------------------------------
// mx_pair_kernel: many rows per group.  A persistent cluster of two CTAs per
// 256 weight rows x up to 192 activation rows (cta_group::2: one MMA of M =
// 256 over both SMs, each CTA holding its 128 weight rows, half of the
// activation rows and 128 lanes of the accumulator).  Sharing the activation
// rows is what the FP4 rate asks for: an SM's operands per 256 k are (128 +
// 96) x 128 bytes for 384 cycles of MMA, 75 bytes a cycle, where one CTA
// alone would need 107.
// Bound: a stage of 192 rows takes 401 cycles (MXFP4; NVFP4 415) against the
// 384 of its MMAs, 390 (398) with the loads left out; of 64 rows 325, the
// issuing warp's own latency.  4096 x 4096 x 4096 in 28.1 us (4.9 PFLOP/s).
// Large calls take more than their stages: 4096 x 14336 x 4096, 17 rounds of 16
// stages, 147,000 cycles where 17 x 16 x 401 are 109,000 (start and last epilogue
// 10,000; the rest, 1,600 a unit, is not accounted for), and at the 1000 W limit
// the clock falls to 1.5 GHz, 95 us.
//   warps 0 and 14: bulk-tensor producers, a stage in turn (each CTA loads its
//   own operands; the leader's barrier counts both); one warp alone needs 390
//   cycles for a stage's four copies, as long as its MMAs take;
//   warp 1: tensor memory, and in the leader the MMA issuer;
//   warps 2-13: epilogue, three warps per quarter of the lanes: with two the
//   last unit's, which nothing hides, took 5,300 cycles.
// Where the units do not fill the pairs, a cluster of 2 or 4 pairs shares one
// along K, its sums joined as in mx_stream_kernel.
// Two accumulators of 192 columns: the epilogue of a unit runs beside the MMAs
// of the next.  384 + 24 (NVFP4: 48) columns of scales fit in 512; 256-wide
// accumulators would leave no room for them.
// A unit's rows start at a multiple of 64 rows of their group, so its scales
// start at column 0 or 2 of their tile.
// ---------------------------------------------------------------------------
constexpr int kPairRows = 192, kPairEpiWarps = 12, kPairThreads = 96 + 32 * kPairEpiWarps;

// The units' order.  Grouped, and dense with at least as many activation rows
// as weight rows: all weight tiles of one piece of rows, then the next piece.
// Dense with fewer activation rows (pieces > 0): all pieces of one weight tile,
// so that the larger operand passes through L2 once (512 x 28672 x 4096: 37.5
// -> 34.3 us; the sizes where both fit alike do not change).
struct PairOrder {
    int ntiles, pieces;
    __device__ __forceinline__ int tile(int u) const { return pieces ? u / pieces : u % ntiles; }
    __device__ __forceinline__ RowUnit rows(RowWalk &walk, const Problem &p, int u, int step) const
    {
        if (pieces && u / pieces >= ntiles) return RowUnit{0, 0, 0, 0, 0};
        return walk.at(p, pieces ? u % pieces : u / ntiles, step);
    }
};

template <bool NV> struct PairCfg {
    static constexpr uint32_t kA = 128 * 128, kB = kPairRows / 2 * 128, kS = kStepTiles<NV> * kTileBytes;
    static constexpr uint32_t kStage = kA + kB + 3 * kS;  // scales: own weight rows, and two tile rows of activations
    static constexpr int kStages = (int)((232448u - 1024u - 512u) / kStage);
    static constexpr uint32_t kSmem = kStages * kStage + 512u + 1024u;
    static constexpr uint32_t kSfaCols = kStepTiles<NV> * 4, kSfbCols = kStepTiles<NV> * 8;
    static_assert(2 * kPairRows + kSfaCols + kSfbCols <= 512, "tensor memory");
    static_assert(16 * kStages + 40 <= 256, "barriers");
    static_assert((kPairRows + 3) * 128 * 4 <= kStages * kStage, "the sums of a cluster's CTA");
};

// An arrival on a barrier of either CTA that orders no memory: it says that
// tensor memory has been read (tcgen05.wait::ld and the fence before it order
// that).  As a release it waited for the warp's stores of the outputs, 2,000
// to 3,000 cycles a unit.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// loads into this CTA's shared memory that count on a barrier of either CTA of the pair
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

template <bool NV, typename TOut, bool GATE>
__global__ void __launch_bounds__(kPairThreads, 1)
    mx_pair_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_a,
                   const __grid_constant__ CUtensorMap tmap_a64, const __grid_constant__ CUtensorMap tmap_a32,
                   const __grid_constant__ CUtensorMap tmap_sw, const __grid_constant__ CUtensorMap tmap_sa,
                   const __grid_constant__ Problem p, PairOrder order, int step, int splits, TOut *__restrict__ Y, int inject_stall)
{
    using Cfg = PairCfg<NV>;
    constexpr int STAGES = Cfg::kStages;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *bars = smem + STAGES * Cfg::kStage;
    const uint32_t full = smem_addr(bars), empty = full + 8 * STAGES, acc_full = empty + 8 * STAGES, acc_empty = acc_full + 16,
                   drained = acc_empty + 16;
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(bars + 256);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 260);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the cluster: `splits` pairs, pair z takes part z of K; `pair` and `pairs` count whole clusters
    const uint32_t crank = cluster_rank(), rank = crank & 1u, z = crank >> 1, leader = crank & ~1u;
    const uint16_t both = (uint16_t)(3u << leader);
    const int pair = blockIdx.x / (2 * splits), pairs = gridDim.x / (2 * splits);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; s++) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; b++) {
            mbar_init(acc_full + 8 * b, 1);
            mbar_init(acc_empty + 8 * b, 2 * kPairEpiWarps);  // the epilogue warps of both CTAs
        }
        mbar_init(drained, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr((const void *)tmem_slot)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        pdl_trigger();  // not before: see the allocation's rule in the header of this file
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers and tensor memory are ready
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();  // the activations come from an earlier kernel of the stream
    if (p.E > 0 && blockIdx.x == 0 && warp == 2) check_offsets(p.offsets, p.E, p.T);
    const int steps = stages_of(p.K);
    const int g0 = (int)((int64_t)steps * z / splits), nk = (int)((int64_t)steps * (z + 1) / splits) - g0;  // this pair's stages

    if (warp == 0 || warp == kPairEpiWarps + 2) {
        // ---------------- producers ----------------
        const uint32_t lead = elect_one(), full0 = cluster_addr(full, leader);
        // the two warps take the stages in turn
        const uint32_t turn = warp == 0 ? 0u : 1u;
        uint32_t s = turn, ph = 0, base = 0;  // base: stages before this unit
        bool ok = true, ready = true;
        RowWalk walk;
        walk.begin(p, step);
        for (int u = pair; ok; u += pairs, base += (uint32_t)nk) {
            const RowUnit w = order.rows(walk, p, u, step);
            if (w.count <= 0) break;
            const int n0 = order.tile(u) * 256 + (int)rank * 128;
            const int half = ((w.count + 15) & ~15) / 2, arow = w.row0 + min((int)rank * half, w.count);  // each CTA holds half of the unit's rows
            // the box that holds them, in one copy (three boxes of 32 took a third longer than one of 96)
            const CUtensorMap *tmap_act = half > 64 ? &tmap_a : half > 32 ? &tmap_a64 : &tmap_a32;
            const uint32_t bytes = Cfg::kStage - Cfg::kB + (uint32_t)(half > 64 ? 96 : half > 32 ? 64 : 32) * 128u;
            const int wrow = w.e * p.N + n0;
            // a weight tile row that does not exist: any other will do, its rows are not written
            const int srow = w.e * p.trows_w + min(n0 / kTileRows, p.trows_w - 1);
            for (int g = (int)((base ^ turn) & 1u); g < nk; g += 2) {
                const uint32_t e = empty + 8 * s, fl = full + 8 * s, f = full0 + 8 * s, a0 = smem_addr(smem) + s * Cfg::kStage,
                               s0 = a0 + Cfg::kA + Cfg::kB, now = ph;
                if (!mbar_wait_tested(ready, e, now ^ 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                s += 2;
                if (s >= STAGES) {
                    s -= STAGES;
                    ph ^= 1u;
                }
                ready = mbar_test(empty + 8 * s, ph ^ 1u);
                // fault injection (tests only): the first CTA never fills its first stage
                const bool stall = inject_stall && blockIdx.x == 0 && base == 0 && g == 0;
                const int c0 = (g0 + g) * 128, t0 = (g0 + g) * kStepTiles<NV> * 2;
                if (lead && !stall) {
                    if (rank == 0) mbar_expect_tx(fl, 2 * bytes);
                    tma_load_2d_pair(a0, &tmap_w, c0, wrow, f);
                    tma_load_2d_pair(a0 + Cfg::kA, tmap_act, c0, arow, f);
                    tma_load_3d_pair(s0, &tmap_sw, 0, t0, srow, f);
                    tma_load_3d_pair(s0 + Cfg::kS, &tmap_sa, 0, t0, w.trow, f);
                }
            }
        }
        if (!ok) {
            // loads already issued land within microseconds; they count on the
            // leader's barrier, which may never complete: wait a fixed 2 ms
            const uint64_t t0 = globaltimer();
            while (globaltimer() - t0 < 2000000ull) {
            }
        }
    } else if (warp == 1) {
        if (rank == 0) {
            // ---------------- MMA issuer (leader) ----------------
            const uint32_t lead = elect_one(), sfa = tmem + 2 * kPairRows, sfb = sfa + Cfg::kSfaCols;
            // One stage's copies, then its MMAs, the scales always in the same columns
            // (copies and MMAs of one thread run in order).  Copying the next stage's
            // scales between the MMAs of this one, or two stages' at once, measured
            // 10% slower: the tensor pipe drains at each change between the two.
            uint32_t s = 0, ph = 0, ti = 0;
            bool ok = true, ready = false;
            RowWalk walk;
            walk.begin(p, step);
            for (int u = pair; ok; u += pairs, ti++) {
                const RowUnit w = order.rows(walk, p, u, step);
                if (w.count <= 0) break;
                const uint32_t b = ti & 1u, acc = tmem + b * kPairRows;
                // the epilogue has drained this accumulator
                if (!mbar_wait_all(acc_empty + 8 * b, ((ti >> 1) & 1u) ^ 1u, abort_flag)) break;
                const uint32_t idesc = idesc_fp4(NV, 256, (w.count + 15) & ~15), off2 = (uint32_t)w.off >> 5;
                for (int g = 0; g < nk; g++) {
                    if (!mbar_wait_tested(ready, full + 8 * s, ph, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a0 = smem_addr(smem) + s * Cfg::kStage, b0 = a0 + Cfg::kA, s0 = b0 + Cfg::kB, e = empty + 8 * s;
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                    ready = mbar_test(full + 8 * s, ph);
                    issue_scales<NV, true, 2>(lead, s0, s0 + Cfg::kS, sfa, sfb);
                    issue_mmas<NV, true, 2>(lead, acc, a0, b0, sfa, sfb, off2, idesc, g == 0);
                    commit<true>(lead, e, both);
                }
                if (ok) commit<true>(lead, acc_full + 8 * b, both);
            }
            // every MMA issued has completed before the tensor memory is freed (bounded)
            asm volatile("{ .reg .pred e; setp.ne.b32 e, %1, 0; @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(
                             drained),
                         "r"(lead)
                         : "memory");
            const uint64_t t0 = globaltimer();
            while (!mbar_try_wait(drained, 0) && globaltimer() - t0 < kTimeoutNs) {
            }
            __syncwarp();
        }
    } else {
        // ---------------- epilogue ----------------
        const int q = warp & 3, c_first = ((warp - 2) >> 2) * 32;  // quarter of the lanes; which of each 96 columns
        const uint32_t acc_empty0 = cluster_addr(acc_empty, leader);
        const int64_t ldy = GATE ? p.N / 2 : p.N;
        const float ts_a = p.ts_a ? *p.ts_a : 1.0f;
        uint32_t ti = 0;
        RowWalk walk;
        walk.begin(p, step);
        for (int u = pair;; u += pairs, ti++) {
            const RowUnit w = order.rows(walk, p, u, step);
            if (w.count <= 0) break;
            const uint32_t b = ti & 1u;
            if (!mbar_wait_warp(acc_full + 8 * b, (ti >> 1) & 1u, abort_flag)) break;
            tc_fence_after();
            const int n = order.tile(u) * 256 + (int)rank * 128 + q * 32 + lane;
            const float scale = p.ts_w ? __fmul_rn(ts_a, p.ts_w[w.e]) : ts_a;
#pragma unroll 1
            for (int c0 = c_first; c0 < w.count || c0 == c_first; c0 += kPairEpiWarps * 8) {
                float v[32];
                tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + b * kPairRows + (uint32_t)c0, v);
                if (c0 + kPairEpiWarps * 8 >= w.count) {
                    // this warp has read its part of the accumulator: hand it back
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(acc_empty0 + 8 * b);
                }
                if (splits == 1) {
                    write_columns<TOut, GATE>(v, scale, p.N, Y, ldy, w.row0 + c0, w.count - c0, n, lane);
                } else {
                    // the ring is free: the cluster's only unit has been read by its MMAs
                    float *part = reinterpret_cast<float *>(smem) + c0 * 128 + q * 32 + lane;
#pragma unroll
                    for (int i = 0; i < 32; i++)
                        if (c0 + i < w.count) part[i * 128] = v[i] * scale;
                }
            }
        }
        tc_fence_before();
    }
    __syncwarp();
    __syncthreads();
    if (splits > 1) {
        cluster_sync();  // every CTA's sums are written
        if (warp >= 2 && warp < kPairEpiWarps + 2) {
            RowWalk walk;
            walk.begin(p, step);
            const RowUnit w = order.rows(walk, p, pair, step);
            const int v = warp - 2;
            join_sums<TOut, GATE>(smem_addr(smem), w.count, splits, (int)rank, 2, (kPairEpiWarps / 4) * (int)z + (v >> 2), kPairEpiWarps / 4 * splits,
                                  v & 3, order.tile(pair) * 256 + (int)rank * 128, p.N, Y, w.row0, lane);
        }
        __syncwarp();
    }
    cluster_sync();  // no CTA leaves while another may still signal its barriers or read its sums
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
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

// scale tiles [tile rows][ct tiles] as rows of 256 bytes, read in boxes of `rows` x `tiles` tiles
static bool encode_tiles_map(CUtensorMap *map, const void *base, int64_t trows, int64_t ct, int rows, int tiles)
{
    const EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[3] = {256u, (cuuint64_t)(2 * ct), (cuuint64_t)trows};
    const cuuint64_t strides[2] = {256u, (cuuint64_t)(ct * kTileBytes)};
    const cuuint32_t box[3] = {256u, (cuuint32_t)(2 * tiles), (cuuint32_t)rows};
    const cuuint32_t es[3] = {1u, 1u, 1u};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// pieces of `step` rows that T rows in E groups can make
static int64_t max_pieces(int64_t T, int64_t E, int64_t step) { return E == 0 ? (T + step - 1) / step : T / step + (E < T ? E : T); }

// CTAs that share one unit along K, 1 to 8 of two stages at least: doubled
// while the CTAs have an SM each.  (8 rows, us for 1 / 2 / 4 / 8: 16 units of 32
// stages 13.3 / 9.9 / 7.8 / 7.3, 31 units 13.4 / 10.0 / 8.3 / 8.7.)  Two CTAs to an
// SM gain from two to four (60 units of 56 stages 21.5 / 15.0 / 14.0), as long as
// the clusters fit at once (74 units: 15.9 / 24.1); from one to two they gain
// where the units leave bandwidth over, the longer K the more (80 units: 8.8 / 8.8
// of 16 stages, 14.1 / 12.4 of 32; 112 units 14.5 / 15.4 of 32, 22.7 / 21.5 of 56);
// from four to eight nothing.
static int stream_splits(int64_t units, int64_t steps)
{
    const int64_t sms = sm_count();
    int S = 1;
    for (; S < 8 && 4 * S <= steps; S *= 2) {
        const int64_t ctas = units * 2 * S;
        if (ctas <= sms) continue;
        if (S == 1 && ctas <= 2 * sms && units <= 2 * sms / 5 + steps) continue;
        if (S == 2 && ctas <= 2 * sms - sms / 6) continue;
        break;
    }
    return S;
}

template <bool NV, typename TOut, bool GATE, typename TIn>
static razer_status launch_stream(const TIn *X, const uint8_t *codes_a, const uint8_t *codes_w, Problem p, TOut *Y, cudaStream_t st)
{
    static PerDevice<bool> allowed;
    int dev = 0;
    bool set;
    cudaGetDevice(&dev);
    if (!allowed.get(dev, set, [](bool &ok) {
            return ok = cudaFuncSetAttribute(mx_stream_kernel<NV, TOut, GATE, TIn>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)kStreamSmem) == cudaSuccess;
        }))
        return RAZER_ERR_CUDA;
    CUtensorMap mw, ma, msw, msa;
    const int64_t E = p.E ? p.E : 1, arows = p.E ? tile_rows_grouped(p.T, p.E) : tile_rows(p.T);
    if (!encode_codes_map(&mw, codes_w, p.N * E, p.K, 128) || !encode_tiles_map(&msw, p.tiles_w, E * p.trows_w, p.ct, 1, kStepTiles<NV>))
        return RAZER_ERR_CUDA;
    if (std::is_void<TIn>::value) {
        if (!encode_codes_map(&ma, codes_a, p.T, p.K, kBoxRows) || !encode_tiles_map(&msa, p.tiles_a, arows, p.ct, 1, kStepTiles<NV>))
            return RAZER_ERR_CUDA;
    } else {
        ma = mw;  // not used
        msa = msw;
    }
    const int ntiles = p.trows_w;  // tiles of 128 weight rows; N + 127 may pass 2^31
    const int64_t pieces = max_pieces(p.T, p.E, kStreamRows), units = pieces * ntiles;
    if (units > INT32_MAX - 1024) return RAZER_ERR_SHAPE;
    p.pieces = (int)pieces;
    const int S = stream_splits(units, stages_of(p.K));
    // one CTA (or cluster) a unit, or where they are more, two CTAs an SM that take several
    const int64_t grid = S > 1 ? units * S : std::min<int64_t>(units, 2 * (int64_t)sm_count());
    const int boxes = p.T <= kBoxRows ? 1 : kStreamRows / kBoxRows;
    const int inject = fault_injection_enabled() ? 1 : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kStreamThreads);
    cfg.dynamicSmemBytes = kStreamSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)S;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = S > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, mx_stream_kernel<NV, TOut, GATE, TIn>, mw, ma, msw, msa, p, X, ntiles, S, boxes, Y, inject) != cudaSuccess)
        return RAZER_ERR_CUDA;
    return RAZER_OK;
}

static int64_t rows_per_group(int64_t T, int64_t E) { return E > 0 ? (T + E - 1) / E : T; }

// Rows of a unit (192, or fewer where smaller units need no more rounds over
// the pairs of SMs) and pairs that share one along K (one unit a cluster then).
// A stage's time goes as 220 + rows (4096 x 4096, one round of 16 stages: 8.7 /
// 9.6 / 10.4 us for 64 / 128 / 192 rows, 5 of them the launch), joining the
// sums takes as long as some 8 stages; so 256 rows take 64 at a time (9.2 us, 192
// at a time 10.4), 700 rows 192 (11.0; 128: 13.7, 64: 16.8), and 128 rows x 4096 x
// 14336 take four pairs to a unit (18.0 -> 14.4 us).
struct PairPlan {
    int step, splits;
};
// clusters of 2, 4, 8 CTAs that the device holds at once
struct PairClusters {
    int pairs[3];
};
static PairPlan pair_plan(const Problem &p, int ntiles, const int (&pairs)[3])
{
    const int64_t E = p.E ? p.E : 1, rows = rows_per_group(p.T, p.E), nk = stages_of(p.K);
    PairPlan best = {kPairRows, 1};
    int64_t cost = INT64_MAX;
    for (int i = 0; i < (p.E ? 1 : 3); i++) {
        const int S = 1 << i;
        for (int step = kPairRows; step >= 64; step -= 64) {
            const int64_t units = E * ((rows + step - 1) / step) * ntiles;
            if (S > 1 && (units > pairs[i] || 2 * S > nk)) continue;
            const int64_t c = (units + pairs[i] - 1) / pairs[i] * ((nk + S - 1) / S + (S > 1 ? 8 : 0)) * (220 + step);
            if (c < cost) {
                cost = c;
                best = {step, S};
            }
        }
    }
    return best;
}

template <bool NV, typename TOut, bool GATE>
static razer_status launch_pair(const uint8_t *codes_a, const uint8_t *codes_w, Problem p, TOut *Y, cudaStream_t st)
{
    using Cfg = PairCfg<NV>;
    static PerDevice<PairClusters> resident;
    int dev = 0;
    PairClusters clusters_of;
    cudaGetDevice(&dev);
    if (!resident.get(dev, clusters_of, [](PairClusters &c) {
            if (cudaFuncSetAttribute(mx_pair_kernel<NV, TOut, GATE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg::kSmem) != cudaSuccess)
                return false;
            for (int i = 0; i < 3; i++) {
                cudaLaunchConfig_t cfg = {};
                cfg.gridDim = dim3((unsigned)(sm_count() / (2 << i) * (2 << i)));
                cfg.blockDim = dim3(kPairThreads);
                cfg.dynamicSmemBytes = Cfg::kSmem;
                cudaLaunchAttribute attr[1];
                attr[0].id = cudaLaunchAttributeClusterDimension;
                attr[0].val.clusterDim.x = 2u << i;
                attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
                cfg.attrs = attr;
                cfg.numAttrs = 1;
                if (cudaOccupancyMaxActiveClusters(&c.pairs[i], mx_pair_kernel<NV, TOut, GATE>, &cfg) != cudaSuccess || c.pairs[i] < 1) {
                    if (i == 0) return false;
                    (void)cudaGetLastError();
                    c.pairs[i] = 0;  // a partition that holds none: K is not split so far
                }
                c.pairs[i] = std::min(c.pairs[i], sm_count() / (2 << i));
            }
            return true;
        }))
        return RAZER_ERR_CUDA;
    const int(&pairs)[3] = clusters_of.pairs;
    CUtensorMap mw, ma, ma64, ma32, msw, msa;
    const int64_t E = p.E ? p.E : 1, arows = p.E ? tile_rows_grouped(p.T, p.E) : tile_rows(p.T);
    if (!encode_codes_map(&mw, codes_w, p.N * E, p.K, 128) || !encode_codes_map(&ma, codes_a, p.T, p.K, kPairRows / 2) ||
        !encode_codes_map(&ma64, codes_a, p.T, p.K, 64) || !encode_codes_map(&ma32, codes_a, p.T, p.K, 32) ||
        !encode_tiles_map(&msw, p.tiles_w, E * p.trows_w, p.ct, 1, kStepTiles<NV>) ||
        !encode_tiles_map(&msa, p.tiles_a, arows, p.ct, 2, kStepTiles<NV>))
        return RAZER_ERR_CUDA;
    const int ntiles = (p.trows_w + 1) / 2;
    const PairPlan plan = pair_plan(p, ntiles, pairs);
    const int64_t pieces = max_pieces(p.T, p.E, plan.step), units = pieces * ntiles;
    if (units > INT32_MAX - 1024) return RAZER_ERR_SHAPE;
    p.pieces = (int)pieces;
    const PairOrder order = {ntiles, p.E == 0 && p.T < p.N ? (int)pieces : 0};
    const int inject = fault_injection_enabled() ? 1 : 0;
    const int64_t clusters = plan.splits > 1 ? units : std::min<int64_t>(units, pairs[0]);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2u * (unsigned)plan.splits * (unsigned)clusters);
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = Cfg::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2u * (unsigned)plan.splits;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, mx_pair_kernel<NV, TOut, GATE>, mw, ma, ma64, ma32, msw, msa, p, order, plan.step, plan.splits, Y, inject) !=
        cudaSuccess)
        return RAZER_ERR_CUDA;
    return RAZER_OK;
}

// The two kernels at up to 64 rows, us: 33 rows x 4096 x 4096 stream 8.1, pair
// 8.6; 64 rows x 4096 x 14336 13.6 and 18.1, x 28672 x 4096 14.4 and 15.2; 128
// rows 12.2 and 8.6, 19.5 and 18.0, 21.3 and 16.7.
template <bool NV, typename TOut, bool GATE>
static razer_status launch_mx(const uint8_t *codes_a, const uint8_t *codes_w, const Problem &p, TOut *Y, cudaStream_t st)
{
    if (rows_per_group(p.T, p.E) > kStreamRows) return launch_pair<NV, TOut, GATE>(codes_a, codes_w, p, Y, st);
    return launch_stream<NV, TOut, GATE, void>(nullptr, codes_a, codes_w, p, Y, st);
}

template <typename TOut>
static razer_status run_mx_t(bool nv, const void *X, razer_dtype x_dt, const uint8_t *codes_a, const uint8_t *codes_w, const Problem &p, TOut *Y,
                             cudaStream_t st)
{
    if (p.K == 0) {
        const int64_t cols = p.gate ? p.N / 2 : p.N;
        mx_zero_kernel<TOut><<<sm_count() * 4, 256, 0, st>>>(p.offsets, p.E, p.T, cols, Y);
        return last_launch_status();
    }
    if (X) {
        if (x_dt == RAZER_F16) {
            const __half *x = reinterpret_cast<const __half *>(X);
            if (p.gate) return launch_stream<false, TOut, true, __half>(x, nullptr, codes_w, p, Y, st);
            return launch_stream<false, TOut, false, __half>(x, nullptr, codes_w, p, Y, st);
        }
        const __nv_bfloat16 *x = reinterpret_cast<const __nv_bfloat16 *>(X);
        if (p.gate) return launch_stream<false, TOut, true, __nv_bfloat16>(x, nullptr, codes_w, p, Y, st);
        return launch_stream<false, TOut, false, __nv_bfloat16>(x, nullptr, codes_w, p, Y, st);
    }
    if (p.gate) return nv ? launch_mx<true, TOut, true>(codes_a, codes_w, p, Y, st) : launch_mx<false, TOut, true>(codes_a, codes_w, p, Y, st);
    return nv ? launch_mx<true, TOut, false>(codes_a, codes_w, p, Y, st) : launch_mx<false, TOut, false>(codes_a, codes_w, p, Y, st);
}

}  // namespace mx

// whether an online call quantizes inside the product (few rows per group)
bool gemm_mx_fuses(int64_t T, int64_t E) { return mx::rows_per_group(T, E) <= (E > 0 ? mx::kFuseGroupRows : mx::kFuseRows); }

// E = 0: dense (offsets ignored); otherwise W is [E, N, K] and ts_w holds E
// scales.  X: the activations, to be quantized to MXFP4 inside the product
// (gemm_mx_fuses), or NULL: they are packed.  The caller has checked every
// argument; T, N > 0.
razer_status run_gemm_mx(const void *X, razer_dtype x_dt, const uint8_t *codes_a, const uint8_t *tiles_a, const float *ts_a, int64_t T,
                         const int32_t *offsets, int E, const uint8_t *codes_w, const uint8_t *tiles_w, const float *ts_w, razer_format fmt, int64_t N, int64_t K, int gate,
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
    p.pieces = 0;  // the launch knows
    if (out_dt == RAZER_F32) return mx::run_mx_t<float>(nv, X, x_dt, codes_a, codes_w, p, reinterpret_cast<float *>(Y), st);
    if (out_dt == RAZER_F16) return mx::run_mx_t<__half>(nv, X, x_dt, codes_a, codes_w, p, reinterpret_cast<__half *>(Y), st);
    return mx::run_mx_t<__nv_bfloat16>(nv, X, x_dt, codes_a, codes_w, p, reinterpret_cast<__nv_bfloat16 *>(Y), st);
}

}  // namespace razer
