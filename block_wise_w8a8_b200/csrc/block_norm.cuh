// block_norm.cuh -- the residual update between two blocks, fused: the branch's RMSNorm, its
// gate, the residual scale and sum, then the next block's RMSNorm with scale and shift, with
// BF16 or 4-bit output.
//
//   u = y                                       without post-norm, else
//   u = (y * rstd(y)) (* post_gamma)
//   h' = bf16( res_scale * h + gate[b] * u )    (gate 1 where there is none), b = row / T
//   n  = bf16( ((h' * rstd(h')) (* pre_gamma)) * (1 + scale[b]) + shift[b] )
//   rstd(v) = 1 / sqrt( mean(v^2) + eps )
//
// in FP32, rounded at h' and n alone; the second norm reads h' as it is stored.  The 4-bit
// output is that of the quantizer of fp4.cuh on n, code for code.
//
// Bound by HBM: h and y are read, h' and n written once (8 bytes a value, 6.6 with 4-bit
// output).  W warps share a row and keep its h and y, later h' and n, in registers; the
// sums of squares go through shuffles and shared memory.  The column factors are read
// through L1, which a row's neighbours keep warm.
#pragma once

#include "common.cuh"
#include "fp4.cuh"

namespace w8a8 {
namespace bnorm {

constexpr int kWarps = 8;                        // warps of a CTA
constexpr int kOutBf16 = -1;                     // else fp4::kMx / fp4::kNv

struct Params {
    const uint16_t *h, *y;                       // [M, K] BF16
    const uint16_t *post_gamma, *pre_gamma;      // [K] or null
    const uint16_t *gate, *scale, *shift;        // [M / T, K] or null
    int64_t M, M_pad, K, T;                      // M_pad: M rounded up to 128 for 4-bit output
    float eps, res_scale;
    int32_t post_norm;
    uint16_t *h_out;                             // [M, K], may be h
    uint16_t *n_out;                             // [M, K] (BF16 output)
    uint8_t *codes, *scales;                     // 4-bit output, as the quantizer's
    float *factor;
};

template <int V>
__device__ __forceinline__ void load_row(const uint16_t *p, uint32_t (&w)[V / 2])
{
#pragma unroll
    for (int i = 0; i < V / 8; ++i) {
        const uint4 a = *(reinterpret_cast<const uint4 *>(p) + i);
        w[4 * i] = a.x; w[4 * i + 1] = a.y; w[4 * i + 2] = a.z; w[4 * i + 3] = a.w;
    }
}
template <int V>
__device__ __forceinline__ void load_col(const uint16_t *p, uint32_t (&w)[V / 2])
{
#pragma unroll
    for (int i = 0; i < V / 8; ++i) {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p) + i);
        w[4 * i] = a.x; w[4 * i + 1] = a.y; w[4 * i + 2] = a.z; w[4 * i + 3] = a.w;
    }
}
template <int V>
__device__ __forceinline__ void store_row(uint16_t *p, const uint32_t (&w)[V / 2])
{
#pragma unroll
    for (int i = 0; i < V / 8; ++i)
        *(reinterpret_cast<uint4 *>(p) + i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

template <int V>
__device__ __forceinline__ float squares(const uint32_t (&w)[V / 2])
{
    float a = 0.0f, b = 0.0f;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        a = fmaf(bf16_lo(w[i]), bf16_lo(w[i]), a);
        b = fmaf(bf16_hi(w[i]), bf16_hi(w[i]), b);
    }
    return a + b;
}

// Sum (or maximum) over the W warps of a row; every thread of the CTA takes part.
template <int W>
__device__ __forceinline__ float row_sum(float v, float *s, int warp, uint32_t lane)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (W > 1) {
        if (lane == 0)
            s[warp] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i)
            v += s[warp / W * W + i];
    }
    return v;
}
template <int W>
__device__ __forceinline__ uint32_t row_max(uint32_t v, float *s, int warp, uint32_t lane)
{
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if (W > 1) {
        if (lane == 0)
            s[warp] = __uint_as_float(v);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < W; ++i)
            v = max(v, __float_as_uint(s[warp / W * W + i]));
    }
    return v;
}

__device__ __forceinline__ float rstd_of(float sum, int64_t K, float eps)
{
    return __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sum, static_cast<float>(K)), eps)));
}

// h' of V values.
template <int V>
__device__ __forceinline__ void update(const Params &p, const uint32_t (&h)[V / 2], const uint32_t (&y)[V / 2],
                                       float rstd, int64_t col, int64_t mod, uint32_t (&o)[V / 2])
{
    uint32_t pg[V / 2], g[V / 2];
    if (p.post_gamma != nullptr)
        load_col<V>(p.post_gamma + col, pg);
    if (p.gate != nullptr)
        load_col<V>(p.gate + mod + col, g);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        float u0 = __fmul_rn(bf16_lo(y[i]), rstd), u1 = __fmul_rn(bf16_hi(y[i]), rstd);
        if (p.post_gamma != nullptr) {
            u0 = __fmul_rn(u0, bf16_lo(pg[i]));
            u1 = __fmul_rn(u1, bf16_hi(pg[i]));
        }
        if (p.gate != nullptr) {
            u0 = __fmul_rn(u0, bf16_lo(g[i]));
            u1 = __fmul_rn(u1, bf16_hi(g[i]));
        }
        o[i] = pack_bf16x2(__fmaf_rn(p.res_scale, bf16_lo(h[i]), u0), __fmaf_rn(p.res_scale, bf16_hi(h[i]), u1));
    }
}

// n of V values of h'.
template <int V>
__device__ __forceinline__ void normalise(const Params &p, const uint32_t (&h)[V / 2], float rstd, int64_t col,
                                          int64_t mod, uint32_t (&o)[V / 2])
{
    uint32_t g[V / 2], sc[V / 2], sh[V / 2];
    if (p.pre_gamma != nullptr)
        load_col<V>(p.pre_gamma + col, g);
    if (p.scale != nullptr)
        load_col<V>(p.scale + mod + col, sc);
    if (p.shift != nullptr)
        load_col<V>(p.shift + mod + col, sh);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        float a = __fmul_rn(bf16_lo(h[i]), rstd), b = __fmul_rn(bf16_hi(h[i]), rstd);
        if (p.pre_gamma != nullptr) {
            a = __fmul_rn(a, bf16_lo(g[i]));
            b = __fmul_rn(b, bf16_hi(g[i]));
        }
        if (p.scale != nullptr) {
            a = __fmul_rn(a, __fadd_rn(1.0f, bf16_lo(sc[i])));
            b = __fmul_rn(b, __fadd_rn(1.0f, bf16_hi(sc[i])));
        }
        if (p.shift != nullptr) {
            a = __fadd_rn(a, bf16_lo(sh[i]));
            b = __fadd_rn(b, bf16_hi(sh[i]));
        }
        o[i] = pack_bf16x2(a, b);
    }
}

// kOut: BF16 or a 4-bit format (V = 16).  A row of at most 32 V W P values stays in registers;
// a longer one is read again for each of its passes (kLong).
template <int kOut, int V, int W, int P, bool kLong>
__global__ void __launch_bounds__(kWarps * 32) block_norm_kernel(const Params p)
{
    static_assert(kOut == kOutBf16 || V == 16, "a lane encodes 16 values");
    __shared__ float s_red[3][kWarps];
    asm volatile("griddepcontrol.launch_dependents;");
    const int warp = threadIdx.x >> 5;
    const uint32_t lane = lane_id();
    const int64_t r = static_cast<int64_t>(blockIdx.x) * (kWarps / W) + warp / W;
    const bool live = r < p.M;
    const int64_t np = live ? p.K / V : 0;       // pieces of the row
    const int64_t b0 = (warp % W) * 32 + lane;
    constexpr int64_t kStep = W * 32;
    constexpr int64_t kChunk = kStep * P;
    const int64_t at = r * p.K;
    const int64_t mod = live ? r / p.T * p.K : 0;
    uint32_t h[P][V / 2], y[P][V / 2];           // y becomes h', h becomes n

    // the branch's sum of squares
    float rstd = 1.0f, sum = 0.0f;
    for (int64_t c = 0; c < np; c += kChunk) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int64_t b = b0 + c + i * kStep;
            if (b < np) {
                load_row<V>(p.y + at + b * V, y[i]);
                if (!kLong)
                    load_row<V>(p.h + at + b * V, h[i]);
            }
        }
        if (!p.post_norm)
            continue;
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (b0 + c + i * kStep < np)
                sum += squares<V>(y[i]);
    }
    if (p.post_norm)
        rstd = rstd_of(row_sum<W>(sum, s_red[0], warp, lane), p.K, p.eps);

    // h', and its sum of squares
    sum = 0.0f;
    for (int64_t c = 0; c < np; c += kChunk) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int64_t b = b0 + c + i * kStep;
            if (b < np) {
                if (kLong) {
                    load_row<V>(p.y + at + b * V, y[i]);
                    load_row<V>(p.h + at + b * V, h[i]);
                }
                uint32_t o[V / 2];
                update<V>(p, h[i], y[i], rstd, b * V, mod, o);
                store_row<V>(p.h_out + at + b * V, o);
                sum += squares<V>(o);
#pragma unroll
                for (int j = 0; j < V / 2; ++j)
                    y[i][j] = o[j];
            }
        }
    }
    rstd = rstd_of(row_sum<W>(sum, s_red[1], warp, lane), p.K, p.eps);

    // n, and for kNv its largest magnitude
    fp4::Row row{};
    uint32_t top = 0;
    if (kOut == kOutBf16 || kOut == fp4::kNv || !kLong) {
        for (int64_t c = 0; c < np; c += kChunk) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int64_t b = b0 + c + i * kStep;
                if (b < np) {
                    if (kLong)
                        load_row<V>(p.h_out + at + b * V, y[i]);
                    normalise<V>(p, y[i], rstd, b * V, mod, h[i]);
                    if constexpr (kOut == kOutBf16)
                        store_row<V>(p.n_out + at + b * V, h[i]);
                    else
                        top = max(top, fp4::amax16(h[i]));
                }
            }
        }
    }
    if constexpr (kOut != kOutBf16) {
        if (kOut == fp4::kNv) {
            row = fp4::row_of(row_max<W>(top, s_red[2], warp, lane));
            if (live && b0 == 0)
                p.factor[r] = row.factor;
        }
        if (r >= p.M_pad)
            return;
        const int64_t KT = fp4::scale_tiles(p.K, kOut);
        constexpr int kPer = kOut == fp4::kNv ? 4 : 8;
        const int64_t nb_pad = KT * kPer;
        for (int64_t c = 0; c < nb_pad; c += kChunk) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int64_t b = b0 + c + i * kStep;
                const bool in = b < np;
                if (kLong && in) {
                    load_row<V>(p.h_out + at + b * V, y[i]);
                    normalise<V>(p, y[i], rstd, b * V, mod, h[i]);
                }
                uint32_t m = in ? fp4::amax16(h[i]) : 0;
                if (kOut == fp4::kMx)
                    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
                uint32_t byte = 0;
                if (in) {
                    const uint2 o = fp4::encode16<kOut>(h[i], m, row, byte);
                    *reinterpret_cast<uint2 *>(p.codes + r * (p.K / 2) + b * 8) = o;
                }
                const uint32_t word = fp4::gather_scales<kOut>(byte);
                if (b < nb_pad && fp4::stores_scales<kOut>(b))
                    *reinterpret_cast<uint32_t *>(p.scales + fp4::scale_word(r, b / kPer, KT)) = word;
            }
        }
    }
}

} // namespace bnorm
} // namespace w8a8
