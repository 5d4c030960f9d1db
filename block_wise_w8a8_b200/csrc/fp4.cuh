// fp4.cuh -- microscaled 4-bit floating point: quantization of BF16 rows and the values
// back.
//
// Elements are E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign), two to a byte, the even
// element in the low half.  Two formats of block scale along K:
//
//   kMx  32 elements share a power of two (OCP Microscaling Formats 1.0, MXFP4):
//          e = max(floor(log2 amax) - 2, -127), byte e + 127 (0 for an all-zero block),
//          code = e2m1(v 2^-e), round to nearest even, saturating.
//        A block with an infinity or a NaN has byte 255 (NaN) and codes 0.
//   kNv  16 elements share an E4M3 number s, and every row has an FP32 factor:
//          A = max(row's amax, 2^-100),  factor = fl(A / 2688)        (2688 = 6 * 448)
//          s = e4m3(448 amax / A),  code = e2m1(2688 v / (s A)), 0 where s is 0.
//        A row with an infinity or a NaN has factor NaN, scales and codes 0.
//
// The value of a code is code * scale (* factor).  The row factor lets a row's largest
// block use E4M3's whole range whatever the row's size; it depends on no other row, so a
// row's codes are the same in every batch.
//
// Both formats' quotients are taken exactly as written, although nothing is divided:
//   kMx  v 2^-e is exact in FP32.
//   kNv  448 amax has 11 significant bits, A 8; 2688 v has 13 and s A 12.  A rounding
//        boundary of E4M3 is j 2^i with odd j < 32, of E2M1 with odd j <= 7, so a quotient
//        off the boundary is off by 2^-13 (scale) or 2^-14.9 (code) of itself at least: two
//        different whole numbers, the larger below 32 * 2^8 or 7 * 2^12, differ by one.  The
//        products with reciprocals below are within 2^-21 of the quotients (three roundings
//        and two reciprocals good to one unit in the last place).  Rounded to 17 significant
//        bits (scale), or to a multiple of 2^-17 (code: below 9.1, the most where a scale is
//        rounded down to E4M3's smallest; boundaries from 0.25 to 5), they lie on a boundary
//        only if the quotient does, and on the same side otherwise.
//        (A negative value below 2^-18 of the unit becomes +0 on the way, others -0.)
//
// Scales lie as tcgen05 block-scaled products read them: 512-byte tiles of 128 rows x 4
// scales along K, tile [row / 128][block / 4], byte 16 (row % 32) + 4 (row % 128 / 32) +
// block % 4.  Rows and blocks past the end of the matrix have scale 0.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace w8a8 {
namespace fp4 {

constexpr int kMx = 0;
constexpr int kNv = 1;
constexpr int kWarps = 8;                       // warps of a quantizer CTA
constexpr float kTiny = 7.888609052210118e-31f; // 2^-100
constexpr float kRowDiv = 2688.0f;

// 512-byte scale tiles along K: 4 scales of 32 (kMx) or 16 (kNv) elements.
__host__ __device__ constexpr int64_t scale_tiles(int64_t K, int fmt)
{
    return fmt == kMx ? (K + 127) / 128 : (K + 63) / 64;
}

// Byte offset of row r's first four scales; the next four are 512 bytes on.
__device__ __forceinline__ int64_t scale_row(int64_t r, int64_t KT)
{
    return (r >> 7) * KT * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

// Eight FP32 numbers -> eight E2M1 codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8])
{
    uint32_t o;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(o)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return o;
}

// Eight E2M1 codes -> four packed FP16 pairs (exact).
__device__ __forceinline__ void from_e2m1x8(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// The E4M3 byte nearest a >= 0, and the FP32 value of an E4M3 byte.
__device__ __forceinline__ uint32_t to_e4m3(float a)
{
    uint16_t o;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(o) : "f"(0.0f), "f"(a));
    return o & 0xFFu;
}
__device__ __forceinline__ float from_e4m3(uint32_t byte)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(byte)));
    float f;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(h));
    return f;
}

// a rounded to 17 significant bits, and 1 / a to one unit in the last place (a normal, > 0).
__device__ __forceinline__ float round17(float a)
{
    return __uint_as_float((__float_as_uint(a) + 0x40u) & ~0x7Fu);
}
__device__ __forceinline__ float reciprocal(float a)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
    return r;
}

// Largest BF16 magnitude pattern among 8 values (4 packed words), in the low 16 bits.
__device__ __forceinline__ uint32_t amax8(const uint32_t (&w)[4])
{
    const uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
    return max(m & 0xFFFFu, m >> 16);
}

// What a row's factor and its blocks' scales are taken from (kNv), given the row's largest
// magnitude pattern.
struct Row {
    float top;        // A; unused for kMx, like the rest
    float to_scale;   // 448 / A
    float to_code;    // 2688 / A
    bool bad;         // the row holds an infinity or a NaN
    __device__ __forceinline__ float factor() const      // what is stored
    {
        return bad ? __uint_as_float(0x7FC00000u) : __fdiv_rn(top, kRowDiv);
    }
};
__device__ __forceinline__ Row row_of(uint32_t amax_bits)
{
    Row r;
    r.bad = amax_bits >= 0x7F80u;
    r.top = r.bad ? 1.0f : fmaxf(__uint_as_float(amax_bits << 16), kTiny);
    const float q = reciprocal(r.top * (1.0f / 4096.0f));       // 4096 / A, a normal number
    r.to_scale = 0.109375f * q;
    r.to_code = 0.65625f * q;
    return r;
}

// Where a lane holds 8 consecutive values (a warp's loads and stores of BF16 are then 512
// contiguous bytes), 2 (kNv) or 4 (kMx) neighbouring lanes share a block.  Lane order =
// order along K.
template <int kFmt>
constexpr int kBlockLanes = kFmt == kMx ? 4 : 2;

// The largest magnitude of the lane's block, from its own values'.
template <int kFmt>
__device__ __forceinline__ uint32_t block_amax(uint32_t m)
{
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    return kFmt == kMx ? max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2)) : m;
}

// The scale byte of a block, given its largest magnitude pattern m, and what its values are
// multiplied by before they are rounded to E2M1; codes are 0 where `zero`.
struct Unit {
    uint32_t byte;
    float mult;
    bool zero;
};
template <int kFmt>
__device__ __forceinline__ Unit unit_of(uint32_t m, const Row &row)
{
    Unit u;
    if (kFmt == kMx) {
        const uint32_t e = m >> 7;                       // exponent field of the largest
        u.zero = e == 255u;
        u.byte = u.zero ? 255u : (e > 2u ? e - 2u : 0u);
        u.mult = u.zero ? 0.0f : __uint_as_float((254u - u.byte) << 23);
    } else {
        u.zero = row.bad;
        u.byte = u.zero ? 0u : to_e4m3(round17(__uint_as_float(m << 16) * row.to_scale));
        u.mult = u.byte == 0u ? 0.0f : row.to_code * reciprocal(from_e4m3(u.byte));
    }
    return u;
}

// Codes of 8 values (4 packed BF16 pairs).
template <int kFmt>
__device__ __forceinline__ uint32_t codes8(const uint32_t (&w)[4], const Unit &u)
{
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = make_float2(bf16_lo(w[i]), bf16_hi(w[i])), m2 = make_float2(u.mult, u.mult);
        float2 q;
        if (kFmt == kMx) {
            q = __fmul2_rn(x, m2);
        } else {                 // to a multiple of 2^-17: FP32's step between 64 and 128
            q = __ffma2_rn(x, m2, make_float2(96.0f, 96.0f));
            q = __fadd2_rn(q, make_float2(-96.0f, -96.0f));
        }
        v[2 * i] = q.x;
        v[2 * i + 1] = q.y;
    }
    return u.zero ? 0u : e2m1x8(v);
}
template <int kFmt>
__device__ __forceinline__ uint32_t encode8(const uint32_t (&w)[4], uint32_t m, const Row &row, uint32_t &byte)
{
    const Unit u = unit_of<kFmt>(m, row);
    byte = u.byte;
    return codes8<kFmt>(w, u);
}

// Offset of the scale of piece b's block from its row's first, and whether this lane stores
// it.  A byte each: gathering a tile's four into a word first takes two shuffles and more
// instructions than the stores it saves.
template <int kFmt>
__device__ __forceinline__ uint32_t scale_offset(int b)
{
    constexpr int lanes = kBlockLanes<kFmt>;
    return static_cast<uint32_t>(b / (4 * lanes)) * 512 + (b / lanes & 3);
}
template <int kFmt>
__device__ __forceinline__ bool stores_scale(int b)
{
    return (b & (kBlockLanes<kFmt> - 1)) == 0;
}

// Codes and block scale of a lane's piece b of a row, from its values and their largest
// magnitude m; every lane of the warp takes part, `in` (b < np) or not.  codes and scales:
// the row's.
template <int kFmt>
__device__ __forceinline__ void store_piece(uint8_t *codes, uint8_t *scales, int b, bool in, int np_pad, const Row &row,
                                            const uint32_t (&w)[4], uint32_t m)
{
    m = block_amax<kFmt>(in ? m : 0);
    uint32_t byte = 0;
    if (in)
        *reinterpret_cast<uint32_t *>(codes + static_cast<uint32_t>(b) * 4) = encode8<kFmt>(w, m, row, byte);
    if (stores_scale<kFmt>(b) && b < np_pad)
        scales[scale_offset<kFmt>(b)] = static_cast<uint8_t>(byte);
}
// Pieces of 8 values of a row with its last scale tile filled up.
template <int kFmt>
__device__ __forceinline__ int pieces_padded(int64_t KT)
{
    return static_cast<int>(KT) * 4 * kBlockLanes<kFmt>;
}

// Places for a value of each of W warps, read by fours from 3 on.
template <int W>
constexpr int kSlots = W < 3 ? W : (W + 3) / 4 * 4;

// Largest magnitude pattern over the W warps of a row (s[kSlots<W>], zeros behind W, if W > 1
// in shared memory); every thread of the row takes part.
template <int W>
__device__ __forceinline__ uint32_t row_top(uint32_t v, uint32_t *s, int warp, uint32_t lane)
{
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if (W > 1) {
        if (lane == 0)
            s[warp] = v;
        __syncthreads();
        if constexpr (W == 2) {
            v = max(s[0], s[1]);
        } else {
#pragma unroll
            for (int i = 0; i < W; i += 4) {
                const uint4 f = *reinterpret_cast<const uint4 *>(s + i);
                v = max(v, max(max(f.x, f.y), max(f.z, f.w)));
            }
        }
    }
    return v;
}

// Programmatic launch (without the attribute both are nothing): a grid reads and writes
// nothing before the grids ahead of it are complete; the next one may be set up from the time
// that every CTA has said so, late in its work: CTAs that only wait take places and are dealt
// out unevenly (quantize + dequantize 1000 x 2048, said at the start: 6.7 us for 4.9).
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;"); }

// By one thread of a CTA whose wait gave up, at the CTA's end: copies in flight land before its
// shared memory is released, for it may be another CTA's next.  They need microseconds, this
// waits a millisecond.
__device__ __forceinline__ void hold_smem()
{
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 1000000ull)
        ;
}

struct QParams {
    const uint16_t *x;       // [rows, K] BF16
    int64_t rows, rows_pad;  // rows_pad: rows rounded up to 128 (the scale tiles' rows)
    int64_t K;               // a multiple of 32
    uint8_t *codes;          // [rows, K / 2]
    uint8_t *scales;         // [rows_pad / 128, KT, 512]
    float *factor;           // [rows] (kNv)
};

__device__ __forceinline__ void load8(const uint16_t *p, uint32_t (&w)[4])
{
    const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p));
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
}

// Scales of rows past the end: zeros, by CTA `cta` of `ctas`.
__device__ __forceinline__ void zero_scales(uint8_t *scales, int64_t rows, int64_t rows_pad, int64_t KT, int64_t cta,
                                            int64_t ctas)
{
    for (int64_t r = rows + cta; r < rows_pad; r += ctas)
        for (int64_t t = threadIdx.x; t < KT; t += blockDim.x)
            *reinterpret_cast<uint32_t *>(scales + scale_row(r, KT) + t * 512) = 0;
}

// Few rows, or rows too long for the ring below.  W warps, one row; a lane holds up to P
// pieces of 8 values in registers, so the row is read once when K <= 256 W P (longer rows are
// read again, from L2, for the codes).  CTAs past the last row clear its tile's scales.
template <int kFmt, int W, int P>
__global__ void __launch_bounds__(W * 32) quantize_kernel(const QParams p)
{
    __shared__ __align__(16) uint32_t s_top[W];
    wait_for_previous();
    const int warp = threadIdx.x >> 5;
    const uint32_t lane = lane_id();
    const int64_t r = blockIdx.x;
    const int np = static_cast<int>(p.K / 8);
    const int64_t KT = scale_tiles(p.K, kFmt);
    if (r >= p.rows) {
        zero_scales(p.scales, r, r + 1, KT, 0, 1);
        return;
    }
    const int np_pad = pieces_padded<kFmt>(KT);
    const int b0 = warp * 32 + static_cast<int>(lane);
    constexpr int kStep = W * 32;
    const uint16_t *xr = p.x + r * p.K;
    uint32_t w[P][4], m[P];
    uint32_t top = 0;
    const bool once = np <= kStep * P;
    if (kFmt == kNv || once) {
        for (int c = 0; c < np; c += kStep * P) {
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (b0 + c + i * kStep < np)
                    load8(xr + static_cast<size_t>(b0 + c + i * kStep) * 8, w[i]);
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (b0 + c + i * kStep < np) {
                    m[i] = amax8(w[i]);
                    top = max(top, m[i]);
                }
        }
    }
    Row row{};
    if (kFmt == kNv) {
        row = row_of(row_top<W>(top, s_top, warp, lane));
        if (threadIdx.x == 0)
            p.factor[r] = row.factor();
    }
    let_next_start();
    uint8_t *codes = p.codes + r * (p.K / 2), *scales = p.scales + scale_row(r, KT);
    for (int c = 0; c < np_pad; c += kStep * P) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int b = b0 + c + i * kStep;
            if (!once && b < np) {
                load8(xr + static_cast<size_t>(b) * 8, w[i]);
                m[i] = amax8(w[i]);
            }
            store_piece<kFmt>(codes, scales, b, b < np, np_pad, row, w[i], m[i]);
        }
    }
}

// Bytes into shared memory, completion counted on `bar`; 16-byte aligned, whole 16 bytes.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// Many rows.  CTAs of W warps stay, take every gridDim.x-th row, and have the next rows copied
// into a ring in shared memory (a bulk copy each) while they code: with a CTA a row the loads,
// the arithmetic and the stores of the few CTAs that fit a SM hardly overlap (16384 x 4096
// nvfp4: 49 us).  Then the instructions bound it (ncu: 72% of the issue slots at 15 a value),
// so a lane takes 16 consecutive values, a whole block (kNv) or half of one: what a block costs
// is paid half as often as with 8.  Up to kStreamPieces of them, K <= 1024 W.
constexpr int kStreamPieces = 2;
constexpr int kStreamWarps = 32;                 // warps a SM
// Two rows a CTA hide the copies: 16384 x 4096 nvfp4 30.4 us with 2, 32.4 with 6 and more,
// mxfp4 29.5 and 30.5 (64 to 1024 values a row: alike); the reads of a deeper ring only crowd
// the writes.
constexpr int kRing = 2;
template <int W>
struct StreamTail {                              // behind the ring
    alignas(16) uint32_t top[2][kSlots<W>];      // by row parity
    uint64_t full[kRing];
    int abort;
};

// How a ring ends when a wait for a row gives up: the flag goes up in front of a block barrier,
// and behind it thread 0, finding it up, fills no slot again, for the copy into this one may
// still be in flight and its barrier's phase open.  The rows from there on are worked on as
// they are, so that every warp reaches every barrier; their waits give up at once.  Last,
// thread 0 holds the shared memory (hold_smem).
template <int kFmt, int W>
__global__ void __launch_bounds__(W * 32, kStreamWarps / W) quantize_stream_kernel(const QParams p)
{
    constexpr int P = kStreamPieces;
    extern __shared__ __align__(128) uint8_t ring[];
    const uint32_t row_bytes = static_cast<uint32_t>(p.K) * 2;
    StreamTail<W> &sm = *reinterpret_cast<StreamTail<W> *>(ring + kRing * row_bytes);
    const int warp = threadIdx.x >> 5;
    const uint32_t lane = lane_id();
    const int np = static_cast<int>(p.K / 16);
    const int64_t KT = scale_tiles(p.K, kFmt);
    constexpr int kTileBlocks = kFmt == kMx ? 8 : 4;         // pieces of 16 a scale tile
    const int np_pad = static_cast<int>(KT) * kTileBlocks;
    const int b0 = warp * 32 + static_cast<int>(lane);
    constexpr int kStep = W * 32;
    const bool stores = kFmt == kNv || (lane & 1) == 0;
    const uint32_t scale_at = static_cast<uint32_t>(b0 / kTileBlocks) * 512 + (kFmt == kNv ? b0 & 3 : b0 / 2 & 3);
    // the order in which a lane reads its two 16-byte halves: 8 neighbouring lanes then cover
    // all of the shared memory's banks
    const uint32_t first = lane >> 2 & 1;
    volatile int *abort = &sm.abort;

    auto fetch = [&](int64_t r, int s) {
        mbar_arrive_expect_tx(&sm.full[s], row_bytes);
        bulk_load(ring + static_cast<size_t>(s) * row_bytes, p.x + r * p.K, row_bytes, &sm.full[s]);
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < kRing; ++s)
            mbar_init(&sm.full[s], 1);
        for (int i = W; i < kSlots<W>; ++i)
            sm.top[0][i] = sm.top[1][i] = 0;
        sm.abort = 0;
        fence_barrier_init();
    }
    wait_for_previous();
    if (threadIdx.x == 0) {
        int64_t r = blockIdx.x;
        for (int s = 0; s < kRing && r < p.rows; ++s, r += gridDim.x)
            fetch(r, s);
    }
    __syncthreads();
    int s = 0, par = 0;
    uint32_t phase = 0;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x, par ^= 1) {
        if (r + gridDim.x >= p.rows)
            let_next_start();
        mbar_wait(&sm.full[s], phase, abort);
        const uint8_t *slot = ring + static_cast<size_t>(s) * row_bytes;
        uint32_t w[P][2][4], m[P];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            m[i] = 0;
            if (b0 + i * kStep < np) {
#pragma unroll
                for (uint32_t h = 0; h < 2; ++h) {
                    const uint4 v = ld_shared_v4(slot + (b0 + i * kStep) * 32 + ((first ^ h) << 4));
                    w[i][h][0] = v.x; w[i][h][1] = v.y; w[i][h][2] = v.z; w[i][h][3] = v.w;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if (b0 + i * kStep < np)
                m[i] = max(amax8(w[i][0]), amax8(w[i][1]));
            top = max(top, m[i]);
        }
        Row row{};
        if (kFmt == kNv) {
            row = row_of(row_top<W>(top, sm.top[par], warp, lane));
            if (threadIdx.x == 0)
                p.factor[r] = row.factor();
        } else if (W > 1) {
            __syncthreads();
        }
        if (W == 1)
            __syncwarp();
        // every thread has read the slot
        if (threadIdx.x == 0 && r + static_cast<int64_t>(kRing) * gridDim.x < p.rows && !*abort)
            fetch(r + static_cast<int64_t>(kRing) * gridDim.x, s);
        uint8_t *codes = p.codes + r * (p.K / 2), *scales = p.scales + scale_row(r, KT);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int b = b0 + i * kStep;
            if (kFmt == kMx)
                m[i] = max(m[i], __shfl_xor_sync(0xFFFFFFFFu, m[i], 1));
            Unit u{};
            if (b < np) {
                u = unit_of<kFmt>(m[i], row);
                const uint32_t c0 = codes8<kFmt>(w[i][0], u), c1 = codes8<kFmt>(w[i][1], u);
                *reinterpret_cast<uint2 *>(codes + static_cast<uint32_t>(b) * 8) =
                    first == 0 ? make_uint2(c0, c1) : make_uint2(c1, c0);
            }
            if (stores && b < np_pad)
                scales[scale_at + i * (kStep / kTileBlocks * 512)] = static_cast<uint8_t>(u.byte);
        }
        if (++s == kRing) {
            s = 0;
            phase ^= 1;
        }
    }
    zero_scales(p.scales, p.rows, p.rows_pad, KT, blockIdx.x, gridDim.x);
    if (threadIdx.x == 0 && *abort)
        hold_smem();
}

// y [rows, K] BF16 = the values the codes stand for: fl(code * scale) is exact, the product
// with the row factor is rounded to FP32, the result once more to BF16.  A lane takes 8
// values; a warp kDeqPieces runs of 256 consecutive ones of a row.
struct DParams {
    const uint8_t *codes;
    const uint8_t *scales;
    const float *factor;
    int64_t rows, K;
    uint16_t *y;
};
constexpr int kDeqPieces = 4;

template <int kFmt>
__global__ void __launch_bounds__(kWarps * 32) dequantize_kernel(const DParams p)
{
    wait_for_previous();
    const int lane = static_cast<int>(lane_id());
    const int64_t np = p.K / 8;
    const int64_t per_row = (np + 32 * kDeqPieces - 1) / (32 * kDeqPieces);
    const int64_t KT = scale_tiles(p.K, kFmt);
    const int64_t g = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (g >= p.rows * per_row)
        return;
    const int64_t r = g / per_row;
    const int64_t b0 = (g - r * per_row) * (32 * kDeqPieces) + lane;
    const float f = kFmt == kNv ? __ldg(p.factor + r) : 1.0f;
    uint32_t c[kDeqPieces], byte[kDeqPieces];
#pragma unroll
    for (int i = 0; i < kDeqPieces; ++i) {
        const int64_t b = b0 + i * 32;
        c[i] = byte[i] = 0;
        if (b < np) {
            c[i] = __ldg(reinterpret_cast<const uint32_t *>(p.codes + r * (p.K / 2) + b * 4));
            byte[i] = __ldg(p.scales + scale_row(r, KT) + scale_offset<kFmt>(static_cast<int>(b)));
        }
    }
    let_next_start();
#pragma unroll
    for (int i = 0; i < kDeqPieces; ++i) {
        const int64_t b = b0 + i * 32;
        if (b >= np)
            return;
        float s;
        if (kFmt == kNv)
            s = from_e4m3(byte[i]);
        else    // 2^(byte - 127); byte 0 is 2^-127, a subnormal, and 255 NaN
            s = byte[i] == 255u ? __uint_as_float(0x7FC00000u)
                                : __uint_as_float(byte[i] == 0u ? 0x00400000u : byte[i] << 23);
        uint32_t q[4], o[4];
        from_e2m1x8(c[i], q);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&q[k]));
            o[k] = pack_bf16x2(v.x * s * f, v.y * s * f);
        }
        *reinterpret_cast<uint4 *>(p.y + r * p.K + b * 8) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

} // namespace fp4
} // namespace w8a8
