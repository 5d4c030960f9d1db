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
// Both formats' quotients are taken exactly as written, although no element is divided:
//   kMx  v 2^-e is exact in FP32.
//   kNv  448 amax and A have 11 and 8 significant bits: their IEEE quotient is an E4M3
//        rounding boundary only if the exact one is.  For the codes, 2688 v has 13 bits and
//        s A 12.  A boundary of E2M1 is j 2^i with odd j <= 7, so a quotient off the
//        boundary is off by 2^-14.9 of itself at least (two different whole numbers, the
//        larger below 7 * 2^12, differ by one).  v * fl(0.65625 * fl(1 / (s A / 4096)))
//        is within 2^-22 of the quotient; rounded to 17 significant bits it lies on a
//        boundary only if the quotient does, and on the same side of it otherwise.
//
// Scales lie as tcgen05 block-scaled products read them: 512-byte tiles of 128 rows x 4
// scales along K, tile [row / 128][block / 4], byte 16 (row % 32) + 4 (row % 128 / 32) +
// block % 4.  Rows and blocks past the end of the matrix have scale 0.
#pragma once

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

// Byte offset, inside its tile, of the four scales of row r.
__device__ __forceinline__ int64_t scale_word(int64_t r, int64_t kt, int64_t KT)
{
    return ((r >> 7) * KT + kt) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

// Two FP32 numbers -> two E2M1 codes in the low byte, the first in its low half.
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

// Largest BF16 magnitude pattern among 8 packed words (16 values), in the low 16 bits.
__device__ __forceinline__ uint32_t amax16(const uint32_t (&w)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    return max(m & 0xFFFFu, m >> 16);
}

// What a row's factor and its blocks' scales are taken from (kNv), given the row's largest
// magnitude pattern.
struct Row {
    float top;        // A; unused for kMx
    float factor;     // what is stored; unused for kMx
    bool bad;         // the row holds an infinity or a NaN (kNv)
};
__device__ __forceinline__ Row row_of(uint32_t amax_bits)
{
    Row r;
    r.bad = amax_bits >= 0x7F80u;
    r.top = r.bad ? 1.0f : fmaxf(__uint_as_float(amax_bits << 16), kTiny);
    r.factor = r.bad ? __uint_as_float(0x7FC00000u) : __fdiv_rn(r.top, kRowDiv);
    return r;
}

// Codes of 16 values (8 packed BF16 pairs) and the scale byte of their block; for kMx the
// magnitude pattern `m` is that of all 32 values of the block (two lanes hold them).
template <int kFmt>
__device__ __forceinline__ uint2 encode16(const uint32_t (&w)[8], uint32_t m, const Row &row, uint32_t &byte)
{
    float mult;
    bool zero;
    if (kFmt == kMx) {
        const uint32_t e = m >> 7;                       // exponent field of the largest
        zero = e == 255u;
        byte = zero ? 255u : (e > 2u ? e - 2u : 0u);
        mult = zero ? 0.0f : __uint_as_float((254u - byte) << 23);
    } else {
        byte = row.bad ? 0u : to_e4m3(__fdiv_rn(__uint_as_float(m << 16) * 448.0f, row.top));
        zero = row.bad;
        const float unit = from_e4m3(byte) * (row.top * (1.0f / 4096.0f));
        mult = byte == 0u ? 0.0f : 0.65625f * __frcp_rn(unit);
    }
    uint2 o;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(w[4 * h + i]) * mult;
            v[2 * i + 1] = bf16_hi(w[4 * h + i]) * mult;
        }
        if (kFmt == kNv) {
#pragma unroll
            for (int i = 0; i < 8; ++i)                  // 17 significant bits
                v[i] = __uint_as_float((__float_as_uint(v[i]) + 0x40u) & ~0x7Fu);
        }
        const uint32_t c = zero ? 0u : e2m1x8(v);
        if (h == 0)
            o.x = c;
        else
            o.y = c;
    }
    return o;
}

// One scale byte a lane (each lane holds 16 consecutive values, lane order = order along
// K) -> the four scales of a tile's row in one word, on the lanes that store it: every
// fourth lane (kNv), every eighth (kMx, where two lanes share a block).
template <int kFmt>
__device__ __forceinline__ uint32_t gather_scales(uint32_t byte)
{
    constexpr uint32_t kFull = 0xFFFFFFFFu;
    constexpr int step = kFmt == kNv ? 1 : 2;
    uint32_t v = byte | (__shfl_down_sync(kFull, byte, step) << 8);
    return v | (__shfl_down_sync(kFull, v, 2 * step) << 16);
}
template <int kFmt>
__device__ __forceinline__ bool stores_scales(int64_t block16)
{
    return (block16 & (kFmt == kNv ? 3 : 7)) == 0;
}

struct QParams {
    const uint16_t *x;       // [rows, K] BF16
    int64_t rows, rows_pad;  // rows_pad: rows rounded up to 128 (the scale tiles' rows)
    int64_t K;               // a multiple of 32
    uint8_t *codes;          // [rows, K / 2]
    uint8_t *scales;         // [rows_pad / 128, KT, 512]
    float *factor;           // [rows] (kNv)
};

__device__ __forceinline__ void load16(const uint16_t *p, uint32_t (&w)[8])
{
    const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p));
    const uint4 b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
}

// W warps share a row; a lane holds up to P pieces of 16 values of it in registers, so the
// row is read once when K <= 512 W P (longer rows are read again, from L2, for the codes).
template <int kFmt, int W, int P>
__global__ void __launch_bounds__(kWarps * 32) quantize_kernel(const QParams p)
{
    __shared__ uint32_t s_top[kWarps];
    asm volatile("griddepcontrol.launch_dependents;");
    const int warp = threadIdx.x >> 5;
    const int lane = static_cast<int>(lane_id());
    const int64_t r = static_cast<int64_t>(blockIdx.x) * (kWarps / W) + warp / W;
    const int64_t nb = p.K / 16;
    const int64_t KT = scale_tiles(p.K, kFmt);
    const int64_t nb_pad = KT * (kFmt == kNv ? 4 : 8);
    const int64_t b0 = (warp % W) * 32 + lane;
    constexpr int64_t kStep = W * 32;
    const bool live = r < p.rows;
    const uint16_t *xr = p.x + r * p.K;
    uint32_t w[P][8];
    uint32_t m[P];
    uint32_t top = 0;
    const bool once = nb <= kStep * P;
    if (live && (kFmt == kNv || once)) {
        for (int64_t c = 0; c < nb; c += kStep * P) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int64_t b = b0 + c + i * kStep;
                if (b < nb)
                    load16(xr + b * 16, w[i]);
            }
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int64_t b = b0 + c + i * kStep;
                m[i] = b < nb ? amax16(w[i]) : 0;
                top = max(top, m[i]);
            }
        }
    }
    Row row{};
    if (kFmt == kNv) {
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        if (W > 1) {
            if (lane == 0)
                s_top[warp] = top;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < W; ++i)
                top = max(top, s_top[warp / W * W + i]);
        }
        row = row_of(top);
        if (live && b0 == 0)
            p.factor[r] = row.factor;
    }
    if (r >= p.rows_pad)
        return;
    for (int64_t c = 0; c < nb_pad; c += kStep * P) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int64_t b = b0 + c + i * kStep;
            const bool in = live && b < nb;
            if (!once && in) {
                load16(xr + b * 16, w[i]);
                m[i] = amax16(w[i]);
            }
            uint32_t mm = in ? m[i] : 0;
            if (kFmt == kMx)
                mm = max(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, 1));
            uint32_t byte = 0;
            if (in) {
                const uint2 o = encode16<kFmt>(w[i], mm, row, byte);
                *reinterpret_cast<uint2 *>(p.codes + r * (p.K / 2) + b * 8) = o;
            }
            const uint32_t word = gather_scales<kFmt>(byte);
            if (b < nb_pad && stores_scales<kFmt>(b))
                *reinterpret_cast<uint32_t *>(p.scales + scale_word(r, b / (kFmt == kNv ? 4 : 8), KT)) = word;
        }
    }
}

// y [rows, K] BF16 = the values the codes stand for: fl(code * scale) is exact, the product
// with the row factor is rounded to FP32, the result once more to BF16.  A lane takes 16
// values; a warp 512 consecutive ones of a row.
struct DParams {
    const uint8_t *codes;
    const uint8_t *scales;
    const float *factor;
    int64_t rows, K;
    uint16_t *y;
};

template <int kFmt>
__global__ void __launch_bounds__(kWarps * 32) dequantize_kernel(const DParams p)
{
    const int lane = static_cast<int>(lane_id());
    const int64_t nb = p.K / 16;
    const int64_t per_row = (nb + 31) / 32;
    const int64_t KT = scale_tiles(p.K, kFmt);
    const int64_t total = p.rows * per_row;
    const int64_t g = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (g >= total)
        return;
    const int64_t r = g / per_row;
    const int64_t b = (g - r * per_row) * 32 + lane;
    if (b >= nb)
        return;
    const uint2 c = __ldg(reinterpret_cast<const uint2 *>(p.codes + r * (p.K / 2) + b * 8));
    const int64_t sb = kFmt == kNv ? b : b / 2;
    const uint32_t byte = __ldg(p.scales + scale_word(r, sb / 4, KT) + (sb & 3));
    float s, f;
    if (kFmt == kNv) {
        s = from_e4m3(byte);
        f = __ldg(p.factor + r);
    } else {
        // 2^(byte - 127); byte 0 is 2^-127, a subnormal, and 255 NaN
        s = byte == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);
        f = 1.0f;
    }
    uint32_t o[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t q[4];
        from_e2m1x8(h == 0 ? c.x : c.y, q);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&q[i]));
            o[4 * h + i] = pack_bf16x2(v.x * s * f, v.y * s * f);
        }
    }
    uint4 *dst = reinterpret_cast<uint4 *>(p.y + r * p.K + b * 16);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

} // namespace fp4
} // namespace w8a8
