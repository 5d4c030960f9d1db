// fp4_gemm.cuh -- products of two microscaled 4-bit matrices on the block-scaled tensor
// cores (tcgen05.mma kind::mxf4 / kind::mxf4nvf4):
//
//   y[m, n] = bf16( xf[m] wf[n] sum_b sx[m, b] sw[n, b] sum_{k in block b} cx[m, k] cw[n, k] + bias[n] )
//
// with FP32 accumulation over all of K in tensor memory; the tensor core applies both block
// scales, the epilogue the row factors (formats in fp4.cuh; kMx has no row factors) and
// the bias, and rounds once to BF16.
//
// Operands are read as the quantizer writes them: codes [rows, K / 2] by TMA with 128-byte
// swizzle, 256 elements of K (128 bytes a row) a pipeline stage; scales as whole 512-byte
// tiles, copied on from shared to tensor memory (tcgen05.cp) in front of the products that
// use them.  Past the end of K the TMA fills codes with zeros, and the scales of the last
// partial tile are zeros in memory.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "fp4.cuh"
#include "gemm.cuh"
#include "norm.cuh"

namespace w8a8 {
namespace fp4 {

constexpr int kSliceK = 256;                             // elements of K a stage
__host__ __device__ constexpr int scale_tiles_a_slice(int fmt) { return fmt == kMx ? 2 : 4; }
__host__ __device__ constexpr int scale_slice_bytes(int fmt) { return scale_tiles_a_slice(fmt) * 512; }

// A tile on its way to L2 alone.  The weight's first ones are asked for before the wait for the
// grids ahead: L2 is where writes and reads meet, so they may even be still at work on it.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap *map, int32_t c0, int32_t c1)
{
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1)
                 : "memory");
}

struct GemmParams {
    int64_t M, N, K;
    int32_t slices;              // K slices, ceil(K / 256)
    int32_t num_tm, num_tn;      // tiles along M and N
    // Pair kernel: units 0 .. num_full - 1 are tiles; each tile after them is two units, its
    // halves along N.
    int32_t num_full, num_units;
    const float *xf;             // [M] row factors of x (kNv)
    const float *wf;             // [N] row factors of w (kNv)
    const uint16_t *bias;        // [N] BF16 or null
    uint16_t *y;                 // [M, N] BF16
};

// Instruction descriptor of the block-scaled kinds, both operands E2M1 and K-major:
//   bits 4-5 / 29-30 which byte of the scale words B / A use; bits 7-9 / 10-12 A / B format
//   (1 = E2M1); bits 17-22 N >> 3; bit 23 scale type (0 = UE4M3, 1 = UE8M0); bits 27-28
//   M >> 7.
__host__ __device__ constexpr uint32_t idesc_fp4(int m, int n, int fmt, int sf)
{
    return (static_cast<uint32_t>(sf) << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
           ((fmt == kMx ? 1u : 0u) << 23) | (static_cast<uint32_t>(m >> 7) << 27) | (static_cast<uint32_t>(sf) << 29);
}

// One product step of 64 elements of K.  kMx: a scale word holds 4 scales of 32, a step
// uses two of them (the descriptor says which); kNv: it uses all 4 scales of 16.
template <int kFmt, int kCtas>
__device__ __forceinline__ void umma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate)
{
#define W8A8_FP4_MMA(group, kind)                                                          \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                         \
                 "tcgen05.mma.cta_group::" group "." kind " [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d), \
                 "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate))
    if constexpr (kFmt == kMx && kCtas == 1)
        W8A8_FP4_MMA("1", "kind::mxf4.block_scale.scale_vec::2X");
    else if constexpr (kFmt == kMx)
        W8A8_FP4_MMA("2", "kind::mxf4.block_scale.scale_vec::2X");
    else if constexpr (kCtas == 1)
        W8A8_FP4_MMA("1", "kind::mxf4nvf4.block_scale.scale_vec::4X");
    else
        W8A8_FP4_MMA("2", "kind::mxf4nvf4.block_scale.scale_vec::4X");
#undef W8A8_FP4_MMA
}

// Shared-memory matrix descriptors in two words, so that a step's only arithmetic is on the
// low one: the address >> 4 (bit 16: a leading offset of 1, unused).  High words: operands in
// 128-byte rows, swizzled, 8-row groups 1024 bytes apart; scale tiles of 32 rows of 16 bytes,
// not swizzled, 8-row groups 128 bytes apart.
constexpr uint32_t kOperandHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kScaleHi = (128u >> 4) | (1u << 14);
__device__ __forceinline__ uint32_t operand_lo(const void *p) { return (smem_u32(p) >> 4) | (1u << 16); }
__device__ __forceinline__ uint64_t desc_of(uint32_t lo, uint32_t hi)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}

// 512-byte scale tile, shared -> tensor memory: its 32 rows of 16 bytes to lanes 0-31 (and the
// same to lanes 32-63, 64-95, 96-127) of 4 columns.
template <int kCtas>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t lo)
{
    const uint64_t d = desc_of(lo, kScaleHi);
    if constexpr (kCtas == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d));
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d));
}

// v xf wf + bias for a sum v and its row's and column's factors (kNv), rounded at the product of
// the factors and at the result.  The quantizer's factors lie between 2^-112 and 2^117, so their
// product may leave FP32's normal range where the result does not (rows of 2^-90 times a weight
// of 2^-30), and a zero sum would meet an infinity.  v then takes one factor after the other.
// Both are above 1 or both below 2^-14 at such a place, and |v| is 0 or at least 2^-20: v wf
// overflows, or loses bits, only where the result does.  A warp tests the range of its factors
// once (up to 2% of the time of many tokens, none of few; tested at each output 10 to 40%); an
// output depends on its own v and factors alone.
__device__ __forceinline__ bool normal_range(float p)
{
    return fabsf(p) >= 1.17549435e-38f && fabsf(p) <= 3.40282347e38f;
}
__device__ __forceinline__ float scaled(float v, float xf, float wf, float bias)
{
    const float p = xf * wf;
    return normal_range(p) ? fmaf(v, p, bias) : fmaf(v * wf, xf, bias);
}
// Whether every product of one of the warp's factors a with one of its factors b is in the
// normal range (false where one is negative or NaN).
__device__ __forceinline__ bool normal_products(uint32_t a_min, uint32_t a_max, uint32_t b_min, uint32_t b_max)
{
    const float lo = __uint_as_float(__reduce_min_sync(0xFFFFFFFFu, a_min)) * __uint_as_float(__reduce_min_sync(0xFFFFFFFFu, b_min));
    const uint32_t am = __reduce_max_sync(0xFFFFFFFFu, a_max), bm = __reduce_max_sync(0xFFFFFFFFu, b_max);
    return max(am, bm) < 0x7F800000u && normal_range(lo) && normal_range(__uint_as_float(am) * __uint_as_float(bm));
}

// One lane of the converged warp.  The tcgen05 and TMA instructions below are issued under
// this predicate: the compiler then takes the code for one thread's and keeps operands in
// uniform registers.  Issued by a thread picked with lane == 0, each took about 60 cycles,
// 17 a slice against the 512 cycles of its products.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// ------------------------------------------------------------------ pairs of CTAs
// Tile 256 x 256, two CTAs of a cluster together (cta_group::2): each holds 128 rows of x and
// 128 rows of w in shared memory and the accumulator of its 128 rows of y x all 256
// columns in its tensor memory; the even CTA's MMA thread issues the products for both.
// A slice then costs each SM 32 KB of codes and 3 KB (kMx) or 6 KB (kNv) of scales for 128 x
// 256 x 256 products.  One thread of each CTA loads its own half (signalling the even CTA's
// barrier), the epilogue warps of each store their 128 rows.
//
// kTma: four epilogue warps, 64 columns at a time through shared memory to TMA stores.
// Otherwise (N not a multiple of 8, or y not 16-byte aligned, where no TMA store can go) the
// rows of y start at any even address and are stored two bytes a lane, which takes more
// instructions; eight warps share them, two to the 32 rows of tensor memory that a warp may
// read, 32 columns at a time (1000 x 2016 x 8191: 18 us, with four warps 30; with N = 8192 and
// TMA 14.8).  With TMA eight warps are slower, 427 us for 407 at 16384 x 4096 x 16384.
//
// Tensor memory: two accumulators of 256 columns and the scales do not fit in 512 columns,
// so the accumulators share columns: one at 0, the other ending where the scales begin.
// The warps that read the shared columns read them first, into registers, and then the next
// tile's products start, so only that first read is not overlapped.  A slice's scales are
// copied over those of the slice before the last, whose products have then completed:
// tcgen05.cp is ordered before the products issued after it, but not after those before it.
//
// The tiles of a last, partial round are cut in half along N when the halves fit in one
// round: 256 x 4096 x 4096, 16 tiles on 74 pairs, 11.1 -> 8.9 us; 4096^3 (mxfp4), 3.5 rounds
// in place of 4, 33.9 -> 32.2 us.  With kTma only.
//
// 16384 x 4096 x 16384: 393 to 411 us in a burst (81 to 84% of four times the BF16 rate), 456 to
// 511 back to back; 8192^3 184 us (90%), mxfp4 175 (95%).  Bound by the products and by the power
// limit that sets their clock, in a single call too (%clock64 against %globaltimer in a copy of
// the kernel: 1.32 GHz in the burst, 1.08 back to back; mxfp4 1.38 and 1.14).  A tile of 16
// slices takes 9340 cycles: 525 a slice (mxfp4 513; 512 at the full rate) and 940 in which the
// next tile waits for the shared columns.  4096^3 takes 41,000 cycles at 1.5 GHz: 3700 up to
// the first slice, 34,400 for 3.5 tiles, 2600 for the last epilogue.
constexpr int kPairStages = 5;
constexpr int kPairGroup = 8;                // M tiles of a raster group

template <bool kTma>
struct PairEpi {
    static constexpr int kWarps = kTma ? 4 : 8;
    static constexpr int kParts = kWarps / 4;            // warps that share 32 rows
    static constexpr int kWidth = 256 / kParts;          // columns of a warp
    static constexpr int kChunk = kTma ? 64 : 32;        // columns a step
    static constexpr int kThreads = 64 + 32 * kWarps;
};

template <int kFmt, bool kTma>
struct alignas(1024) PairSmem {
    using E = PairEpi<kTma>;
    uint8_t a[kPairStages][128 * 128];
    uint8_t b[kPairStages][128 * 128];
    uint8_t sfa[kPairStages][scale_slice_bytes(kFmt)];
    uint8_t sfb[kPairStages][2][scale_slice_bytes(kFmt)];
    alignas(1024) uint8_t out[E::kWarps][32 * E::kChunk * 2];   // per epilogue warp: 32 rows
    float col[E::kWarps][2][E::kWidth];      // per epilogue warp: row factors of w, bias
    uint64_t full[kPairStages];              // both CTAs' bytes (the even CTA's)
    uint64_t empty[kPairStages];
    uint64_t tfull[2];
    uint64_t tshared;                        // shared columns read (the even CTA's)
    uint64_t tdrained[2];                    // accumulator read (the even CTA's)
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort;
};
template <int kFmt, bool kTma>
constexpr size_t kPairSmemBytes = sizeof(PairSmem<kFmt, kTma>) + 1024;

// Tensor memory columns of the pair kernel: SFA and SFB of two slices at the end, by slice
// parity, and the second accumulator before them.
__host__ __device__ constexpr uint32_t pair_sf_cols(int fmt) { return 12u * scale_tiles_a_slice(fmt); }
__host__ __device__ constexpr uint32_t pair_acc1(int fmt) { return 512u - 2 * pair_sf_cols(fmt) - 256u; }

__device__ __forceinline__ uint32_t map_to(uint32_t saddr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}
// Arrives on a barrier of either CTA.  Nothing written to memory is handed over (the tensor
// memory loads before it have completed), so the release is left at its default scope, the
// CTA: at cluster scope it waits for this thread's outstanding stores, over 1000 cycles.
__device__ __forceinline__ void arrive_remote(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// TMA load into this CTA's shared memory that signals a barrier of the pair's even CTA.
__device__ __forceinline__ void tma_load_pair(void *dst, const CUtensorMap *map, uint32_t bar, int32_t c0, int32_t c1)
{
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
                 : "memory");
}
// Arrives on the same barrier of both CTAs when this thread's products have completed.
__device__ __forceinline__ void commit_pair(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     smem_u32(bar)),
                 "h"(static_cast<uint16_t>(3))
                 : "memory");
}

// Unit u: its tile, and which half of it along N (-1: all of it).
__device__ __forceinline__ void pair_unit(int u, const GemmParams &p, int &tm, int &tn, int &half)
{
    half = -1;
    int t = u;
    if (u >= p.num_full) {
        t = p.num_full + ((u - p.num_full) >> 1);
        half = (u - p.num_full) & 1;
    }
    const int per_group = kPairGroup * p.num_tn;
    const int group = t / per_group;
    const int first = group * kPairGroup;
    const int gsz = min(p.num_tm - first, kPairGroup);
    const int local = t - group * per_group;
    tm = first + local % gsz;
    tn = local / gsz;
}

// 32 rows x 32 BF16 of a warp's staging buffer (gemm::stage_off) to y, one column a lane; row
// pointers by addition, four in turn.
__device__ __forceinline__ void store_rows(uint16_t *y, int64_t N, const uint8_t *out, int rows, bool in, int lane)
{
    const uint8_t *src[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        src[k] = out + (lane & 7) * 2 + (((lane >> 3) ^ k) << 4);
    uint16_t v[32];
#pragma unroll
    for (int r = 0; r < 32; ++r)
        v[r] = *reinterpret_cast<const uint16_t *>(src[(r >> 1) & 3] + r * 64);
    if (!in)
        return;
    uint16_t *d[4] = {y, y + N, y + 2 * N, y + 3 * N};
    if (rows == 32) {
#pragma unroll
        for (int r = 0; r < 32; ++r) {
            *d[r & 3] = v[r];
            d[r & 3] += 4 * N;
        }
    } else {
#pragma unroll
        for (int r = 0; r < 32; ++r) {
            if (r < rows)
                *d[r & 3] = v[r];
            d[r & 3] += 4 * N;
        }
    }
}

template <int kFmt, bool kTma>
__global__ void __launch_bounds__(PairEpi<kTma>::kThreads, 1)
    gemm_pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                     const __grid_constant__ CUtensorMap tmXs, const __grid_constant__ CUtensorMap tmWs,
                     const __grid_constant__ CUtensorMap tmY, const GemmParams p)
{
    constexpr int kTiles = scale_tiles_a_slice(kFmt);
    constexpr uint32_t kSfBytes = scale_slice_bytes(kFmt);
    // bytes of a slice a CTA loads: 128 rows of x, 128 (half a tile: 64) of w, and their scales
    constexpr uint32_t kSliceBytes = 2 * 128 * 128 + 3 * kSfBytes;
    constexpr uint32_t kHalfBytes = 128 * 128 + 64 * 128 + 2 * kSfBytes;
    extern __shared__ uint8_t smem_raw[];
    using E = PairEpi<kTma>;
    using S = PairSmem<kFmt, kTma>;
    S &sm = *reinterpret_cast<S *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);
    const uint32_t lane = lane_id();
    const uint32_t rank = norm::cluster_rank();
    volatile int *abort = &sm.abort;
    const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
    const int num_units = p.num_units;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kPairStages; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        mbar_init(&sm.tfull[0], 1);
        mbar_init(&sm.tfull[1], 1);
        mbar_init(&sm.tshared, 2 * 4);
        mbar_init(&sm.tdrained[0], 2 * E::kWarps);
        mbar_init(&sm.tdrained[1], 2 * E::kWarps);
        mbar_init(&sm.mma_done, 1);
        sm.abort = 0;
        fence_barrier_init();
        prefetch_tensormap(&tmX);
        prefetch_tensormap(&tmW);
        prefetch_tensormap(&tmXs);
        prefetch_tensormap(&tmWs);
        if (kTma)
            prefetch_tensormap(&tmY);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem_base)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    norm::cluster_barrier();     // both CTAs' barriers are initialised and their TMEM allocated
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    // The operands may come from the quantizer launched before: nothing below reads them
    // before that grid has completed.
    asm volatile("griddepcontrol.wait;" ::: "memory");

    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer
        {
            uint32_t it = 0;
            bool ok = true;
            for (int t = pair; ok && t < num_units; t += pairs) {
                int tm, tn, cut;
                pair_unit(t, p, tm, tn, cut);
                const int32_t row_x = tm * 256 + static_cast<int>(rank) * 128;
                const int32_t row_w = tn * 256 + (cut < 0 ? static_cast<int>(rank) * 128 : cut * 128 + static_cast<int>(rank) * 64);
                for (int ks = 0; ks < p.slices; ++ks, ++it) {
                    const uint32_t s = it % kPairStages, ph = (it / kPairStages) & 1;
                    if (!gemm::gemm_wait(&sm.empty[s], ph ^ 1, abort)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        if (rank == 0)
                            mbar_arrive_expect_tx(&sm.full[s], 2 * (cut < 0 ? kSliceBytes : kHalfBytes));
                        const uint32_t bar = map_to(smem_u32(&sm.full[s]), 0);
                        tma_load_pair(sm.a[s], &tmX, bar, ks * 128, row_x);
                        tma_load_pair(sm.b[s], &tmW, bar, ks * 128, row_w);
                        // scale maps count in 8-byte units: 64 a tile
                        tma_load_pair(sm.sfa[s], &tmXs, bar, ks * (kTiles * 64), row_x >> 7);
                        tma_load_pair(sm.sfb[s][0], &tmWs, bar, ks * (kTiles * 64), tn * 2 + (cut < 0 ? 0 : cut));
                        if (cut < 0) {
                            tma_load_pair(sm.b[s] + 64 * 128, &tmW, bar, ks * 128, row_w + 64);
                            tma_load_pair(sm.sfb[s][1], &tmWs, bar, ks * (kTiles * 64), tn * 2 + 1);
                        }
                    }
                    __syncwarp();
                }
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        if (rank == 0) {
            // One thread issues everything; a slice's 17 instructions and its two waits have to
            // fit the 512 cycles of its products, so ring positions and descriptors are counted
            // on, not computed.
            if (elect_one()) {
                const uint32_t a0 = operand_lo(sm.a[0]), b0 = operand_lo(sm.b[0]);
                const uint32_t fa0 = smem_u32(sm.sfa[0]) >> 4, fb0 = smem_u32(sm.sfb[0][0]) >> 4;
                uint32_t i = 0, it = 0;
                uint32_t s = 0, ph = 0;                              // slice it in the ring
                uint32_t s2 = kPairStages - 2, ph2 = 1;              // slice it - 2
                bool ok = true;
                for (int t = pair; ok && t < num_units; t += pairs, ++i) {
                    const bool whole = t < p.num_full;
                    // tile i - 2 has left this accumulator, tile i - 1 the columns both use (with
                    // kTma the second implies the first: all warps arrive there, tile by tile)
                    if (i > 1 && !gemm::gemm_wait(&sm.tdrained[i & 1], ((i >> 1) - 1) & 1, abort))
                        break;
                    if (i > 0 && !gemm::gemm_wait(&sm.tshared, (i - 1) & 1, abort))
                        break;
                    tc_fence_after();
                    const uint32_t d = tmem + (i & 1) * pair_acc1(kFmt);
                    for (int ks = 0; ks < p.slices; ++ks, ++it) {
                        // the products of slice it - 2 have read the scales that this one replaces
                        if ((it >= 2 && !gemm::gemm_wait(&sm.empty[s2], ph2, abort)) ||
                            !gemm::gemm_wait(&sm.full[s], ph, abort)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t sfa = tmem + 512 - (1 + (it & 1)) * pair_sf_cols(kFmt);
                        const uint32_t sfb = sfa + 4 * kTiles;
                        const uint32_t fa = fa0 + s * (kSfBytes >> 4), fb = fb0 + s * (2 * kSfBytes >> 4);
                        const uint32_t a = a0 + s * (128 * 128 >> 4), b = b0 + s * (128 * 128 >> 4);
#pragma unroll
                        for (int j = 0; j < kTiles; ++j) {
                            copy_scales<2>(sfa + 4 * j, fa + (512 >> 4) * j);
                            copy_scales<2>(sfb + 8 * j, fb + (512 >> 4) * j);
                            if (whole)
                                copy_scales<2>(sfb + 8 * j + 4, fb + (kSfBytes >> 4) + (512 >> 4) * j);
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int j = kFmt == kMx ? k >> 1 : k;
                            const int sf = kFmt == kMx ? (k & 1) * 2 : 0;
                            const uint32_t id = whole ? idesc_fp4(256, 256, kFmt, sf) : idesc_fp4(256, 128, kFmt, sf);
                            umma_fp4<kFmt, 2>(d, desc_of(a + 2 * k, kOperandHi), desc_of(b + 2 * k, kOperandHi), id,
                                              sfa + 4 * j, sfb + 8 * j, (ks | k) != 0);
                        }
                        commit_pair(&sm.empty[s]);
                        if (ks == p.slices - 1)
                            commit_pair(&sm.tfull[i & 1]);
                        if (++s == kPairStages) {
                            s = 0;
                            ph ^= 1;
                        }
                        if (++s2 == kPairStages) {
                            s2 = 0;
                            ph2 ^= 1;
                        }
                    }
                }
                // every product issued here completes before tensor memory is released
                asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                                 smem_u32(&sm.mma_done))
                             : "memory");
                volatile int no_abort = 0;
                mbar_wait(&sm.mma_done, 0, &no_abort, 100000000ull);
            }
            __syncwarp();
        }
    } else {
        // ---------------------------------------------------------------- epilogue
        const int ew = warp - 2;
        const int quarter = warp & 3;
        const int part = ew >> 2;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + part * E::kWidth;
        const uint32_t shared = map_to(smem_u32(&sm.tshared), 0);
        const uint32_t drained = map_to(smem_u32(&sm.tdrained[0]), 0);
        using Chunk = uint32_t[E::kChunk / 32][32];
        auto load_chunk = [](uint32_t taddr, Chunk &r) {
#pragma unroll
            for (int q = 0; q < E::kChunk / 32; ++q)
                tmem_ld32(taddr + q * 32, r[q]);
        };
        auto wait_chunk = [](Chunk &r) {
#pragma unroll
            for (int q = 0; q < E::kChunk / 32; ++q)
                tmem_wait_ld(r[q]);
        };
        uint8_t *out = sm.out[ew];
        float *wf = sm.col[ew][0], *bias = sm.col[ew][1];
        uint32_t i = 0;
        for (int t = pair; t < num_units; t += pairs, ++i) {
            int tm, tn, cut;
            pair_unit(t, p, tm, tn, cut);
            const int64_t m_w = static_cast<int64_t>(tm) * 256 + rank * 128 + quarter * 32;
            const int64_t m = m_w + lane;
            const int64_t n0 = static_cast<int64_t>(tn) * 256 + (cut > 0 ? 128 : 0) + part * E::kWidth;
            constexpr int kSteps = E::kWidth / E::kChunk;
            const int steps = kTma && cut >= 0 ? kSteps / 2 : kSteps;
            __syncwarp();
            const float xf = kFmt == kNv && m < p.M ? __ldg(p.xf + m) : 1.0f;
            uint32_t wf_min = 0x3F800000u, wf_max = wf_min;
#pragma unroll
            for (int j = 0; j < E::kWidth / 32; ++j) {
                const int64_t n = n0 + j * 32 + lane;
                const float f = kFmt == kNv && n < p.N ? __ldg(p.wf + n) : 1.0f;
                wf[j * 32 + lane] = f;
                wf_min = min(wf_min, __float_as_uint(f));
                wf_max = max(wf_max, __float_as_uint(f));
                bias[j * 32 + lane] =
                    p.bias != nullptr && n < p.N ? __uint_as_float(static_cast<uint32_t>(__ldg(p.bias + n)) << 16) : 0.0f;
            }
            const bool all_plain =
                kFmt != kNv || normal_products(__float_as_uint(xf), __float_as_uint(xf), wf_min, wf_max);
            __syncwarp();
            const uint32_t buf = i & 1;
            if (!gemm::gemm_wait(&sm.tfull[buf], (i >> 1) & 1, abort))
                break;
            tc_fence_after();
            const uint32_t acc = lane_base + buf * pair_acc1(kFmt);
            // The columns that both accumulators use (kNv: 96, kMx: 48) are the last of the lower
            // one and the first of the upper one.  A warp's first steps, from that end (two of 64
            // or three of 32), are read into registers at once; with them the shared columns are
            // free, and with the rest the accumulator.
            static_assert(2 * pair_sf_cols(kFmt) <= 96, "shared columns");
            const bool holds_shared = E::kParts == 1 || part != static_cast<int>(buf);
            auto store_chunk = [&](auto plain, const Chunk &r, int c0) {
                if (kTma && lane == 0)
                    gemm::tma_store_wait_read();
                __syncwarp();
#pragma unroll
                for (int g = 0; g < E::kChunk / 8; ++g) {
                    uint32_t o[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int e = g * 8 + q * 2;
                        const float2 f = *reinterpret_cast<const float2 *>(wf + c0 + e);
                        const float2 b = *reinterpret_cast<const float2 *>(bias + c0 + e);
                        const float v0 = __uint_as_float(r[e >> 5][e & 31]), v1 = __uint_as_float(r[e >> 5][(e & 31) + 1]);
                        if (kFmt != kNv)
                            o[q] = pack_bf16x2(v0 + b.x, v1 + b.y);
                        else if (decltype(plain)::value)
                            o[q] = pack_bf16x2(fmaf(v0, xf * f.x, b.x), fmaf(v1, xf * f.y, b.y));
                        else
                            o[q] = pack_bf16x2(scaled(v0, xf, f.x, b.x), scaled(v1, xf, f.y, b.y));
                    }
                    st_shared_v4(out + (kTma ? lane * 128 + ((g ^ (lane & 7)) << 4) : gemm::stage_off(lane, g)),
                                 make_uint4(o[0], o[1], o[2], o[3]));
                }
                const int64_t nc = n0 + c0;
                if (kTma) {
                    gemm::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && m_w < p.M && nc < p.N)
                        gemm::tma_store_2d(&tmY, out, static_cast<int32_t>(nc), static_cast<int32_t>(m_w));
                } else {
                    __syncwarp();
                    store_rows(p.y + m_w * p.N + nc + lane, p.N, out, static_cast<int>(min(static_cast<int64_t>(32), p.M - m_w)),
                               nc + lane < p.N, static_cast<int>(lane));
                }
            };
            auto column = [&](int step) { return (buf == 0 ? steps - 1 - step : step) * E::kChunk; };
            auto arrive = [&](bool here, uint32_t bar) {
                if (here && lane == 0)
                    arrive_remote(bar);
            };
            auto store_unit = [&](auto plain) {
                if constexpr (kTma) {
                    Chunk r0, r1;
                    load_chunk(acc + column(0), r0);
                    load_chunk(acc + column(1), r1);
                    wait_chunk(r0);
                    wait_chunk(r1);
                    tc_fence_before();
                    __syncwarp();
                    arrive(true, shared);
                    arrive(steps == 2, drained + buf * 8);
                    store_chunk(plain, r0, column(0));
                    if (steps == 4)
                        load_chunk(acc + column(2), r0);
                    store_chunk(plain, r1, column(1));
                    if (steps == 4) {
                        load_chunk(acc + column(3), r1);
                        wait_chunk(r0);
                        wait_chunk(r1);
                        tc_fence_before();
                        __syncwarp();
                        arrive(true, drained + buf * 8);
                        store_chunk(plain, r0, column(2));
                        store_chunk(plain, r1, column(3));
                    }
                } else {
#pragma unroll 1
                    for (int step = 0; step < 4; ++step) {
                        const int c0 = column(step);
                        Chunk r;
                        load_chunk(acc + c0, r);
                        wait_chunk(r);
                        if ((step == 2 && holds_shared) || step == 3) {
                            tc_fence_before();
                            __syncwarp();
                            arrive(true, step == 3 ? drained + buf * 8 : shared);
                        }
                        store_chunk(plain, r, c0);
                    }
                }
            };
            if (all_plain)
                store_unit(std::true_type{});
            else if constexpr (kFmt == kNv)
                store_unit(std::false_type{});
        }
        if (kTma && lane == 0)
            gemm::tma_store_wait_all();
    }
    tc_fence_before();
    __syncthreads();
    // no CTA leaves while its peer may still read its shared memory or signal its barriers
    norm::cluster_barrier();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    }
    // a wait of any thread gave up (the producer may have issued its last loads before that):
    // copies in flight land before shared memory is released
    if (threadIdx.x == 0 && *abort)
        hold_smem();
}

// ------------------------------------------------------------------ few tokens
// y^T: the weight's rows are the 128 rows of a product and BT tokens its columns, so that a
// tile costs the weight's bytes and little else.  One tile a CTA; the K slices are split
// over the S CTAs of a cluster, which add their FP32 partial tiles through distributed
// shared memory in rank order (the result does not depend on timing).  The pipeline takes
// less than half of an SM's shared memory: two CTAs a SM keep all SMs streaming when the
// tiles do not divide among them.
//
// kQuant: x is BF16 and quantized on the way in.  Each CTA codes the slices that it
// multiplies, four warps writing them into the pipeline's stages in the layout that the TMA
// would; the weight's loads run ahead meanwhile.  For a few rows this repeated work costs
// less than a launch of the quantizer and its workspace.
constexpr int kSkinnyThreads = 192;

template <int kFmt, int BT>
struct alignas(1024) SkinnySmem {
    static constexpr int kStageBytes = 128 * 128 + BT * 128 + 2 * scale_slice_bytes(kFmt);
    static constexpr int kStages = BT < 64 ? 4 : 3;
    uint8_t w[kStages][128 * 128];       // after the last product, with x: partial [BT][128] FP32
    uint8_t x[kStages][BT * 128];
    uint8_t sfw[kStages][scale_slice_bytes(kFmt)];
    uint8_t sfx[kStages][scale_slice_bytes(kFmt)];
    uint64_t full[kStages];
    uint64_t empty[kStages];
    uint64_t tfull;
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort;
    uint32_t top[4][4];                  // kQuant: per warp and row, the largest magnitude
    float factor[4];                     // kQuant: row factors
    static_assert(BT * 128 * 4 <= kStages * (128 * 128 + BT * 128), "partial tile does not fit");
};
template <int kFmt, int BT>
constexpr size_t kSkinnySmemBytes = sizeof(SkinnySmem<kFmt, BT>) + 1024;
constexpr int kQuantRows = 4;            // most rows of kQuant

// kQuant, kNv: the row factors, from the rows' largest magnitudes over all of K.  Four warps,
// before the CTA's set-up is complete, so that the loads overlap it.
template <class S>
__device__ __forceinline__ void row_tops(S &sm, const GemmParams &p, const uint16_t *x, int tid, uint32_t lane)
{
    // 4 pieces of 8 values of every row in flight
    uint32_t top[kQuantRows] = {};
    const int64_t pieces = p.K / 8;
    for (int64_t c0 = tid; c0 < pieces; c0 += 4 * 128) {
        uint4 v[kQuantRows][4];
#pragma unroll
        for (int m = 0; m < kQuantRows; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[m][i] = m < p.M && c0 + i * 128 < pieces
                              ? __ldg(reinterpret_cast<const uint4 *>(x + m * p.K) + c0 + i * 128)
                              : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int m = 0; m < kQuantRows; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                top[m] = __vmaxu2(top[m], __vmaxu2(__vmaxu2(v[m][i].x & 0x7FFF7FFFu, v[m][i].y & 0x7FFF7FFFu),
                                                   __vmaxu2(v[m][i].z & 0x7FFF7FFFu, v[m][i].w & 0x7FFF7FFFu)));
    }
#pragma unroll
    for (int m = 0; m < kQuantRows; ++m) {
        const uint32_t t = __reduce_max_sync(0xFFFFFFFFu, max(top[m] & 0xFFFFu, top[m] >> 16));
        if (lane == 0)
            sm.top[tid >> 5][m] = t;
    }
}

// kQuant's four warps: the CTA's slices of x, coded into the stages.  A warp takes one row,
// a lane its 8 values of a slice.
template <int kFmt, class S>
__device__ __forceinline__ void quantize_slices(S &sm, const GemmParams &p, const uint16_t *x, int ks0, int ks1, int r,
                                                uint32_t lane, volatile int *abort)
{
    static_assert(kQuantRows == 4, "a warp a row");
    const int64_t np = p.K / 8;
    const int b = static_cast<int>(lane);
    const bool mine = r < p.M;
    const uint16_t *src = x + r * p.K;
    uint32_t w[4] = {};
    if (mine && static_cast<int64_t>(ks0) * 32 + b < np)
        load8(src + (static_cast<int64_t>(ks0) * 32 + b) * 8, w);
    Row row{};
    if (kFmt == kNv) {
        uint32_t t = 0;
        for (int i = 0; i < 4; ++i)
            t = max(t, sm.top[i][r]);
        row = row_of(t);
        if (b == 0)
            sm.factor[r] = row.factor();
    }
    uint32_t it = 0;
    for (int ks = ks0; ks < ks1; ++ks, ++it) {
        const uint32_t s = it % S::kStages, ph = (it / S::kStages) & 1;
        const bool in = mine && static_cast<int64_t>(ks) * 32 + b < np;
        const uint32_t m = block_amax<kFmt>(in ? amax8(w) : 0);
        uint32_t byte = 0, o = 0;
        if (in)
            o = encode8<kFmt>(w, m, row, byte);
        const int64_t nx = static_cast<int64_t>(ks + 1) * 32 + b;
        if (mine && ks + 1 < ks1 && nx < np)
            load8(src + nx * 8, w);
        if (!gemm::gemm_wait(&sm.empty[s], ph ^ 1, abort))
            break;
        if (mine) {
            // row r of the 128-byte-swizzled tile: 16-byte piece b / 4, XOR the row
            *reinterpret_cast<uint32_t *>(sm.x[s] + r * 128 + (((b >> 2) ^ r) << 4) + (b & 3) * 4) = o;
            if (stores_scale<kFmt>(b))
                sm.sfx[s][r * 16 + scale_offset<kFmt>(b)] = static_cast<uint8_t>(byte);
        }
        gemm::fence_proxy_async_smem();      // the products read shared memory as the TMA does
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&sm.full[s]);
    }
    // every thread of the epilogue reads the factors
    if (kFmt == kNv)
        named_bar_sync(1, 128);
}

template <int kFmt, int BT, bool kQuant>
__global__ void __launch_bounds__(kSkinnyThreads, 2)
    gemm_skinny_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                       const __grid_constant__ CUtensorMap tmXs, const __grid_constant__ CUtensorMap tmWs,
                       const uint16_t *x, const GemmParams p)
{
    using S = SkinnySmem<kFmt, BT>;
    constexpr int kTiles = scale_tiles_a_slice(kFmt);
    constexpr int kStages = S::kStages;
    constexpr uint32_t kTxBytes =
        kQuant ? 128 * 128 + scale_slice_bytes(kFmt) : static_cast<uint32_t>(S::kStageBytes);
    // the accumulator, and the scales of each stage
    constexpr uint32_t kUsed = BT + kStages * 8 * kTiles;
    constexpr uint32_t kCols = kUsed <= 128 ? 128 : 256;
    static_assert(kUsed <= 256, "two CTAs share a SM's 512 columns");
    extern __shared__ uint8_t smem_raw[];
    S &sm = *reinterpret_cast<S *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);
    const uint32_t lane = lane_id();
    const int rank = static_cast<int>(norm::cluster_rank()), splits = static_cast<int>(norm::cluster_size());
    volatile int *abort = &sm.abort;
    const int tile = static_cast<int>(blockIdx.x) / splits;
    const int tn = tile % p.num_tn, tm = tile / p.num_tn;
    // the rank's slices
    const int ks0 = static_cast<int>(static_cast<int64_t>(p.slices) * rank / splits);
    const int ks1 = static_cast<int>(static_cast<int64_t>(p.slices) * (rank + 1) / splits);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sm.full[s], kQuant ? 5 : 1);
            mbar_init(&sm.empty[s], 1);
        }
        mbar_init(&sm.tfull, 1);
        mbar_init(&sm.mma_done, 1);
        sm.abort = 0;
        fence_barrier_init();
        prefetch_tensormap(&tmW);
        prefetch_tensormap(&tmWs);
        if (!kQuant) {
            prefetch_tensormap(&tmX);
            prefetch_tensormap(&tmXs);
        }
    }
    if (warp == 2 && elect_one()) {
        for (int ks = ks0; ks < min(ks1, ks0 + kStages); ++ks) {
            tma_prefetch_2d(&tmW, ks * 128, tn * 128);
            tma_prefetch_2d(&tmWs, ks * (kTiles * 64), tn);
        }
    }
    if (warp == 1) {
        tmem_alloc(&sm.tmem_base, kCols);
        tmem_relinquish();
    }
    if (kQuant)
        asm volatile("griddepcontrol.wait;" ::: "memory");
    if (kQuant && kFmt == kNv && warp >= 2)
        row_tops(sm, p, x, static_cast<int>(threadIdx.x) - 64, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    if (!kQuant)
        asm volatile("griddepcontrol.wait;" ::: "memory");
    // The epilogue's thread owns output n and the tokens of this CTA's tile.  Its column's factor
    // and bias are fetched ahead where the factor is looked at before the accumulator is complete.
    float *part = reinterpret_cast<float *>(sm.w);
    const int row = (warp & 3) * 32 + static_cast<int>(lane);
    const int64_t n = static_cast<int64_t>(tn) * 128 + row;
    const int64_t m0 = static_cast<int64_t>(tm) * BT;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(BT), p.M - m0));
    const bool store = warp >= 2 && n < p.N;
    float wf = 1.0f, bias = 0.0f;
    auto fetch_column = [&]() {
        if (store) {
            if (kFmt == kNv)
                wf = __ldg(p.wf + n);
            if (p.bias != nullptr)
                bias = __uint_as_float(static_cast<uint32_t>(__ldg(p.bias + n)) << 16);
        }
    };
    if (!kQuant)
        fetch_column();

    if (warp == 0) {
        uint32_t it = 0;
        for (int ks = ks0; ks < ks1; ++ks, ++it) {
            const uint32_t s = it % kStages, ph = (it / kStages) & 1;
            if (!gemm::gemm_wait(&sm.empty[s], ph ^ 1, abort))
                break;
            if (elect_one()) {
                mbar_arrive_expect_tx(&sm.full[s], kTxBytes);
                tma_load_2d(sm.w[s], &tmW, &sm.full[s], ks * 128, tn * 128);
                tma_load_2d(sm.sfw[s], &tmWs, &sm.full[s], ks * (kTiles * 64), tn);
                if (!kQuant) {
                    tma_load_2d(sm.x[s], &tmX, &sm.full[s], ks * 128, tm * BT);
                    tma_load_2d(sm.sfx[s], &tmXs, &sm.full[s], ks * (kTiles * 64), tm * BT / 128);
                }
            }
            __syncwarp();
        }
        // Nothing is left to fetch: the next grid's first weight tiles may come meanwhile (one
        // token after another, K = 4096, N = 16384: 10.4 us, so 9.4, with the prefetch 8.9;
        // N = 4096 5.7, 4.7, 4.8).  The pair kernel gains as much before another product, but
        // loses it before a quantizer (linear of 128 x 4096 x 16384: 16.5 -> 17.0 us).
        let_next_start();
    } else if (warp == 1) {
        if (elect_one()) {
            const uint32_t w0 = operand_lo(sm.w[0]), x0 = operand_lo(sm.x[0]);
            const uint32_t fw0 = smem_u32(sm.sfw[0]) >> 4, fx0 = smem_u32(sm.sfx[0]) >> 4;
            uint32_t s = 0, ph = 0;
            for (int ks = ks0; ks < ks1; ++ks) {
                if (!gemm::gemm_wait(&sm.full[s], ph, abort))
                    break;
                tc_fence_after();
                // a stage's scales have their own columns: they are free when the stage is
                const uint32_t sfw = tmem + BT + s * (8 * kTiles), sfx = sfw + 4 * kTiles;
                const uint32_t fw = fw0 + s * (scale_slice_bytes(kFmt) >> 4), fx = fx0 + s * (scale_slice_bytes(kFmt) >> 4);
                const uint32_t w = w0 + s * (128 * 128 >> 4), x = x0 + s * (BT * 128 >> 4);
#pragma unroll
                for (int j = 0; j < kTiles; ++j) {
                    copy_scales<1>(sfw + 4 * j, fw + (512 >> 4) * j);
                    copy_scales<1>(sfx + 4 * j, fx + (512 >> 4) * j);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int j = kFmt == kMx ? k >> 1 : k;
                    const uint32_t id = idesc_fp4(128, BT, kFmt, kFmt == kMx ? (k & 1) * 2 : 0);
                    umma_fp4<kFmt, 1>(tmem, desc_of(w + 2 * k, kOperandHi), desc_of(x + 2 * k, kOperandHi), id,
                                      sfw + 4 * j, sfx + 4 * j, ks != ks0 || k != 0);
                }
                umma_commit(&sm.empty[s]);
                if (ks == ks1 - 1)
                    umma_commit(&sm.tfull);
                if (++s == kStages) {
                    s = 0;
                    ph ^= 1;
                }
            }
            // every product issued here completes before tensor memory is released, also where
            // this thread or the epilogue gave up
            umma_commit(&sm.mma_done);
            volatile int no_abort = 0;
            mbar_wait(&sm.mma_done, 0, &no_abort, 100000000ull);
        }
        __syncwarp();
    } else if (kQuant) {
        quantize_slices<kFmt>(sm, p, x, ks0, ks1, warp - 2, lane, abort);
    }
    if (kQuant)
        fetch_column();
    // Whether the products of the warp's columns' factors with the tokens' are all in range.  kQuant
    // has few outputs a thread and tests at each: the factors come late there, and reductions
    // over them would be waited for (4 x 4096 x 4096: 6.3 us for 6.5).
    bool plain = true;
    if (kFmt == kNv && !kQuant && warp >= 2) {
        uint32_t xf_min = 0x3F800000u, xf_max = xf_min;
        for (int t = static_cast<int>(lane); t < tokens; t += 32) {
            const uint32_t f = __float_as_uint(__ldg(p.xf + m0 + t));
            xf_min = min(xf_min, f);
            xf_max = max(xf_max, f);
        }
        plain = normal_products(xf_min, xf_max, __float_as_uint(wf), __float_as_uint(wf));
    }
    auto finish = [&](float v, int t) {
        if (kFmt != kNv)
            v = v + bias;
        else if (kQuant)
            v = scaled(v, sm.factor[t], wf, bias);
        else
            v = fmaf(v, __ldg(p.xf + m0 + t) * wf, bias);
        p.y[(m0 + t) * p.N + n] = static_cast<uint16_t>(pack_bf16x2(v, 0.0f) & 0xFFFFu);
    };
    if (warp >= 2 && gemm::gemm_wait(&sm.tfull, 0, abort)) {
        tc_fence_after();
        const uint32_t acc = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
#pragma unroll 1
        for (int c = 0; c < tokens; c += 16) {
            uint32_t v[16];
            tmem_ld16(acc + c, v);
            tmem_wait_ld(v);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (splits > 1 || !plain)
                    part[(c + i) * 128 + row] = __uint_as_float(v[i]);
                else if (store && c + i < tokens)
                    finish(__uint_as_float(v[i]), c + i);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (splits > 1)
        norm::cluster_barrier();     // every rank's partial tile is in its shared memory
    if (splits > 1 || !plain) {
        // tokens are dealt out to the ranks in equal runs
        const int each = (tokens + splits - 1) / splits;
        const int t1 = min(tokens, (rank + 1) * each);
        if (store && plain && !*abort) {
            // 8 tokens of 4 ranks in flight: a read of another SM's shared memory takes about
            // as long as one of L2
            for (int t0 = rank * each; t0 < t1; t0 += 8) {
                float v[8] = {};
                for (int q0 = 0; q0 < splits; q0 += 4) {
                    float u[4][8];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (q0 + q >= splits)
                            break;
                        const uint32_t base = map_to(smem_u32(part + t0 * 128 + row), static_cast<uint32_t>(q0 + q));
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(u[q][i]) : "r"(base + i * 512));
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (q0 + q >= splits)
                            break;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            v[i] += u[q][i];
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (t0 + i < t1)
                        finish(v[i], t0 + i);
            }
        } else if (kFmt == kNv && !kQuant && store && !*abort) {
            // the same sums, one after the other, where a product of factors is out of range
#pragma unroll 1
            for (int t = rank * each; t < t1; ++t) {
                float v = 0.0f;
#pragma unroll 1
                for (int q = 0; q < splits; ++q) {
                    float u;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                 : "=f"(u)
                                 : "r"(map_to(smem_u32(part + t * 128 + row), static_cast<uint32_t>(q))));
                    v += u;
                }
                p.y[(m0 + t) * p.N + n] =
                    static_cast<uint16_t>(pack_bf16x2(scaled(v, __ldg(p.xf + m0 + t), wf, bias), 0.0f) & 0xFFFFu);
            }
        }
    }
    if (splits > 1)
        norm::cluster_barrier();     // no CTA leaves while another reads its partial tile
    if (warp == 1)
        tmem_dealloc(tmem, kCols);
    // as at the end of the pair kernel
    if (threadIdx.x == 0 && *abort)
        hold_smem();
}

} // namespace fp4
} // namespace w8a8
