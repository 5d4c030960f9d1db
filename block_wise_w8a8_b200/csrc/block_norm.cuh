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
// With BF16 output bound by HBM: h and y are read, h' and n written once (8 bytes a value, 6.6
// with 4-bit output).  W warps share a row and keep its h and y, then h' and n, in registers, P pieces
// of 8 values a lane; the sums of squares go through shuffles and shared memory.  32768 x 4096
// with all factors: 168 us (6.4 TB/s), 193 with NVFP4 and 175 with MXFP4 output (4.6 and 5.0;
// neither HBM nor issue is full there: the latency of a row's reductions, three in turn, at 16
// warps a SM); 1 x 4096 2.3 us.
//
//   stream_kernel  many rows: CTAs stay, take every gridDim.x-th row, and have the next rows'
//                  h and y copied into a ring in shared memory (one bulk copy each) while they
//                  work.  A lane has the same columns in every row: for P <= 2 their factors
//                  stay in registers and are read again when the rows' group b changes; for
//                  more they come from L1 or L2 for each row, ahead of the wait for the row and
//                  of the second sum (4096 x 16384 nvfp4: 160 us; where they are used, 219).
//   row_kernel     few rows, or rows too long for the ring: one row a W warps, straight from
//                  global memory; longer rows are read again for each pass (kLong).
#pragma once

#include "common.cuh"
#include "fp4.cuh"
#include "norm.cuh"

namespace w8a8 {
namespace bnorm {

constexpr int kOutBf16 = -1;                     // else fp4::kMx / fp4::kNv

struct Params {
    const uint16_t *h, *y;                       // [M, K] BF16
    const uint16_t *post_gamma, *pre_gamma;      // [K] or null
    const uint16_t *gate, *scale, *shift;        // [M / T, K] or null
    int64_t M, M_pad, K, T;                      // M_pad: M rounded up to 128 for 4-bit output
    float eps, res_scale;
    int32_t post_norm;
    int32_t stages;                              // stream_kernel: rows in the ring
    uint16_t *h_out;                             // [M, K], may be h
    uint16_t *n_out;                             // [M, K] (BF16 output)
    uint8_t *codes, *scales;                     // 4-bit output, as the quantizer's
    float *factor;
};

__device__ __forceinline__ void unpack4(const uint4 a, uint32_t (&w)[4])
{
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
}
__device__ __forceinline__ uint4 pack4(const uint32_t (&w)[4]) { return make_uint4(w[0], w[1], w[2], w[3]); }
__device__ __forceinline__ float2 pair_of(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }

// The factors of 8 columns in FP32: u = (y rstd) post, n = (h' rstd) pre + shift, with
// post = fl(post_gamma gate) and pre = fl(pre_gamma fl(1 + scale)); 1 and 0 where they are
// left out.
struct Post {
    float2 post[4];
};
struct Pre {
    float2 pre[4], shift[4];
};
// The same as they are read: pairs of BF16.
struct RawPost {
    uint4 gamma, gate;
};
struct RawPre {
    uint4 gamma, scale, shift;
};
__device__ __forceinline__ uint4 raw_factor(const uint16_t *p, int64_t at, uint32_t none)
{
    return p != nullptr ? __ldg(reinterpret_cast<const uint4 *>(p + at)) : make_uint4(none, none, none, none);
}
constexpr uint32_t kOnes = 0x3F803F80u;
__device__ __forceinline__ RawPost fetch_post(const Params &p, int64_t col, int64_t mod)
{
    return {raw_factor(p.post_gamma, col, kOnes), raw_factor(p.gate, mod + col, kOnes)};
}
__device__ __forceinline__ RawPre fetch_pre(const Params &p, int64_t col, int64_t mod)
{
    return {raw_factor(p.pre_gamma, col, kOnes), raw_factor(p.scale, mod + col, 0), raw_factor(p.shift, mod + col, 0)};
}
__device__ __forceinline__ void make_post(const RawPost &raw, Post &c)
{
    uint32_t gamma[4], gate[4];
    unpack4(raw.gamma, gamma);
    unpack4(raw.gate, gate);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c.post[i] = __fmul2_rn(pair_of(gamma[i]), pair_of(gate[i]));
}
__device__ __forceinline__ void make_pre(const RawPre &raw, Pre &c)
{
    uint32_t gamma[4], scale[4], shift[4];
    unpack4(raw.gamma, gamma);
    unpack4(raw.scale, scale);
    unpack4(raw.shift, shift);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        c.pre[i] = __fmul2_rn(pair_of(gamma[i]), __fadd2_rn(make_float2(1.0f, 1.0f), pair_of(scale[i])));
        c.shift[i] = pair_of(shift[i]);
    }
}
__device__ __forceinline__ void load_post(const Params &p, int64_t col, int64_t mod, Post &c)
{
    make_post(fetch_post(p, col, mod), c);
}
__device__ __forceinline__ void load_pre(const Params &p, int64_t col, int64_t mod, Pre &c)
{
    make_pre(fetch_pre(p, col, mod), c);
}

__device__ __forceinline__ void add_squares(const uint32_t (&w)[4], float2 &acc)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = pair_of(w[i]);
        acc = __ffma2_rn(v, v, acc);
    }
}

// Sum over the W warps of a row through s[kSlots<W>] (zeros behind W); every thread of the row
// takes part.
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
        if constexpr (W == 2) {
            v = s[0] + s[1];
        } else {
            v = 0.0f;
#pragma unroll
            for (int i = 0; i < W; i += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(s + i);
                v += (f.x + f.y) + (f.z + f.w);
            }
        }
    }
    return v;
}
__device__ __forceinline__ float rstd_of(float sum, float inv_k, float eps)
{
    return rsqrtf(fmaf(sum, inv_k, eps));
}

// h' of 8 values of h and y; into y.
__device__ __forceinline__ void update(const Post &c, float res_scale, float rstd, const uint32_t (&h)[4],
                                       uint32_t (&y)[4])
{
    const float2 r2 = make_float2(rstd, rstd), s2 = make_float2(res_scale, res_scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 u = __fmul2_rn(__fmul2_rn(pair_of(y[i]), r2), c.post[i]);
        u = __ffma2_rn(s2, pair_of(h[i]), u);
        y[i] = pack_bf16x2(u.x, u.y);
    }
}

// n of 8 values of h'.
__device__ __forceinline__ void normalise(const Pre &c, float rstd, const uint32_t (&h)[4], uint32_t (&n)[4])
{
    const float2 r2 = make_float2(rstd, rstd);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = __ffma2_rn(__fmul2_rn(pair_of(h[i]), r2), c.pre[i], c.shift[i]);
        n[i] = pack_bf16x2(a.x, a.y);
    }
}

// ------------------------------------------------------------------ many rows
constexpr int kMaxRing = 16;             // rows of a ring at most

// Shared memory: the ring, `stages` slots of h and y of a row (4 K bytes), then this.
template <int W>
struct StreamTail {
    static constexpr int kSlots = fp4::kSlots<W>;
    alignas(16) float red[2][2][kSlots]; // by row parity and sum
    alignas(16) uint32_t top[2][kSlots];
    uint64_t full[kMaxRing];
    int abort;
};

constexpr int kStreamWarps = 16;         // warps a SM (128 registers a thread)

template <int kOut, int W, int P>
__global__ void __launch_bounds__(W * 32, P > 2 ? 1 : kStreamWarps / W) stream_kernel(const Params p)
{
    extern __shared__ __align__(128) uint8_t ring[];
    const uint32_t row_bytes = static_cast<uint32_t>(p.K) * 2;
    const int S = p.stages;
    StreamTail<W> &sm = *reinterpret_cast<StreamTail<W> *>(ring + static_cast<size_t>(S) * 2 * row_bytes);
    const int warp = threadIdx.x >> 5;
    const uint32_t lane = lane_id();
    const int np = static_cast<int>(p.K / 8);
    const int b0 = warp * 32 + static_cast<int>(lane);
    const int64_t KT = kOut == kOutBf16 ? 0 : fp4::scale_tiles(p.K, kOut);
    constexpr int kStep = W * 32;
    volatile int *abort = &sm.abort;

    auto fetch = [&](int64_t r, int s) {
        uint8_t *slot = ring + static_cast<size_t>(s) * 2 * row_bytes;
        mbar_arrive_expect_tx(&sm.full[s], 2 * row_bytes);
        fp4::bulk_load(slot, p.y + r * p.K, row_bytes, &sm.full[s]);
        fp4::bulk_load(slot + row_bytes, p.h + r * p.K, row_bytes, &sm.full[s]);
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s)
            mbar_init(&sm.full[s], 1);
        for (int i = W; i < fp4::kSlots<W>; ++i)
            for (int par = 0; par < 2; ++par)
                sm.red[par][0][i] = sm.red[par][1][i] = 0.0f, sm.top[par][i] = 0;
        sm.abort = 0;
        fence_barrier_init();
    }
    fp4::wait_for_previous();
    if (threadIdx.x == 0) {
        int64_t r = blockIdx.x;
        for (int s = 0; s < S && r < p.M; ++s, r += gridDim.x)
            fetch(r, s);
    }
    __syncthreads();

    constexpr bool kKeep = P <= 2;
    Post post[kKeep ? P : 1];
    Pre pre[kKeep ? P : 1];
    const float inv_k = __fdiv_rn(1.0f, static_cast<float>(p.K));
    // the rows' group: its offset in gate, scale and shift, and its end
    int64_t mod = 0, group_end = 0;
    int s = 0, par = 0;
    uint32_t phase = 0;
    for (int64_t r = blockIdx.x; r < p.M; r += gridDim.x, par ^= 1) {
        const bool next_group = r >= group_end;
        if (next_group) {
            const int64_t g = r / p.T;
            mod = g * p.K;
            group_end = (g + 1) * p.T;
        }
        if (kKeep && next_group) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int b = b0 + i * kStep;
                if (b < np) {
                    load_post(p, b * 8, mod, post[kKeep ? i : 0]);
                    load_pre(p, b * 8, mod, pre[kKeep ? i : 0]);
                }
            }
        }
        RawPost raw_post[kKeep ? 1 : P];
        if (!kKeep) {
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (b0 + i * kStep < np)
                    raw_post[kKeep ? 0 : i] = fetch_post(p, (b0 + i * kStep) * 8, mod);
        }
        if (r + gridDim.x >= p.M)
            fp4::let_next_start();
        mbar_wait(&sm.full[s], phase, abort);        // that gives up: see fp4::quantize_stream_kernel
        const uint8_t *slot = ring + static_cast<size_t>(s) * 2 * row_bytes;
        uint32_t y[P][4], h[P][4];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int b = b0 + i * kStep;
            y[i][0] = y[i][1] = y[i][2] = y[i][3] = 0;
            h[i][0] = h[i][1] = h[i][2] = h[i][3] = 0;
            if (b < np) {
                unpack4(ld_shared_v4(slot + b * 16), y[i]);
                unpack4(ld_shared_v4(slot + row_bytes + b * 16), h[i]);
            }
        }
        uint16_t *h_row = p.h_out + r * p.K;
        float rstd = 1.0f;
        if (p.post_norm) {
            float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < P; ++i)
                add_squares(y[i], acc);
            rstd = rstd_of(row_sum<W>(acc.x + acc.y, sm.red[par][0], warp, lane), inv_k, p.eps);
        }
        float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int b = b0 + i * kStep;
            if (b < np) {
                Post &f = post[kKeep ? i : 0];
                if (!kKeep)
                    make_post(raw_post[kKeep ? 0 : i], f);
                update(f, p.res_scale, rstd, h[i], y[i]);
                *reinterpret_cast<uint4 *>(h_row + b * 8) = pack4(y[i]);
                add_squares(y[i], acc);
            }
        }
        RawPre raw_pre[kKeep ? 1 : P];
        if (!kKeep) {
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (b0 + i * kStep < np)
                    raw_pre[kKeep ? 0 : i] = fetch_pre(p, (b0 + i * kStep) * 8, mod);
        }
        if (W == 1)
            __syncwarp();
        rstd = rstd_of(row_sum<W>(acc.x + acc.y, sm.red[par][1], warp, lane), inv_k, p.eps);
        // every thread has read the slot
        if (threadIdx.x == 0 && r + static_cast<int64_t>(S) * gridDim.x < p.M && !*abort)
            fetch(r + static_cast<int64_t>(S) * gridDim.x, s);
        uint32_t top = 0, m[P] = {};
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int b = b0 + i * kStep;
            if (b < np) {
                Pre &f = pre[kKeep ? i : 0];
                if (!kKeep)
                    make_pre(raw_pre[kKeep ? 0 : i], f);
                normalise(f, rstd, y[i], h[i]);
                if constexpr (kOut == kOutBf16)
                    *reinterpret_cast<uint4 *>(p.n_out + r * p.K + b * 8) = pack4(h[i]);
                else
                    top = max(top, m[i] = fp4::amax8(h[i]));
            }
        }
        if constexpr (kOut != kOutBf16) {
            fp4::Row row{};
            if (kOut == fp4::kNv) {
                row = fp4::row_of(fp4::row_top<W>(top, sm.top[par], warp, lane));
                if (threadIdx.x == 0)
                    p.factor[r] = row.factor();
            }
            uint8_t *codes = p.codes + r * (p.K / 2), *scales = p.scales + fp4::scale_row(r, KT);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int b = b0 + i * kStep;
                fp4::store_piece<kOut>(codes, scales, b, b < np, fp4::pieces_padded<kOut>(KT), row, h[i], m[i]);
            }
        }
        if (++s == S) {
            s = 0;
            phase ^= 1;
        }
    }
    if constexpr (kOut != kOutBf16)
        fp4::zero_scales(p.scales, p.M, p.M_pad, KT, blockIdx.x, gridDim.x);
    if (threadIdx.x == 0 && *abort)
        fp4::hold_smem();
}

// ------------------------------------------------------------------ few or long rows
// A row of at most 256 W P values stays in registers; a longer one is read again for each of
// its passes (kLong).  One row a CTA.
template <int kOut, int W, int P, bool kLong>
__global__ void __launch_bounds__(W * 32) row_kernel(const Params p)
{
    __shared__ __align__(16) float s_red[2][W];
    __shared__ __align__(16) uint32_t s_top[W];
    fp4::wait_for_previous();
    const int warp = threadIdx.x >> 5;
    const uint32_t lane = lane_id();
    const int64_t r = blockIdx.x;
    if (kOut != kOutBf16 && r >= p.M) {          // CTAs past the last row clear its tile's scales
        fp4::zero_scales(p.scales, r, r + 1, fp4::scale_tiles(p.K, kOut), 0, 1);
        return;
    }
    const int np = static_cast<int>(p.K / 8);
    const int b0 = warp * 32 + static_cast<int>(lane);
    constexpr int kStep = W * 32;
    constexpr int kChunk = kStep * P;
    const int64_t at = r * p.K;
    const int64_t mod = r / p.T * p.K;
    uint32_t h[P][4], y[P][4];
    // factors of up to two pieces are loaded with the row, ahead of the first reduction
    constexpr bool kAhead = !kLong && P <= 2;
    Post post[kAhead ? P : 1];
    Pre pre[kAhead ? P : 1];
    const float inv_k = __fdiv_rn(1.0f, static_cast<float>(p.K));

    // the branch's sum of squares
    float rstd = 1.0f;
    float2 acc = make_float2(0.0f, 0.0f);
    for (int at_c = 0; at_c < np; at_c += kChunk) {
        if (kLong && !p.post_norm)
            break;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int b = b0 + at_c + i * kStep;
            y[i][0] = y[i][1] = y[i][2] = y[i][3] = 0;
            if (b < np) {
                unpack4(*reinterpret_cast<const uint4 *>(p.y + at + static_cast<size_t>(b) * 8), y[i]);
                if (!kLong) {
                    unpack4(*reinterpret_cast<const uint4 *>(p.h + at + static_cast<size_t>(b) * 8), h[i]);
                }
                if (kAhead) {
                    load_post(p, int64_t{8} * b, mod, post[kAhead ? i : 0]);
                    load_pre(p, int64_t{8} * b, mod, pre[kAhead ? i : 0]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < P; ++i)
            add_squares(y[i], acc);
    }
    if (p.post_norm)
        rstd = rstd_of(row_sum<W>(acc.x + acc.y, s_red[0], warp, lane), inv_k, p.eps);

    // h', and its sum of squares
    acc = make_float2(0.0f, 0.0f);
    for (int at_c = 0; at_c < np; at_c += kChunk) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int b = b0 + at_c + i * kStep;
            if (b < np) {
                if (kLong) {
                    unpack4(*reinterpret_cast<const uint4 *>(p.y + at + static_cast<size_t>(b) * 8), y[i]);
                    unpack4(*reinterpret_cast<const uint4 *>(p.h + at + static_cast<size_t>(b) * 8), h[i]);
                }
                Post &f = post[kAhead ? i : 0];
                if (!kAhead)
                    load_post(p, int64_t{8} * b, mod, f);
                update(f, p.res_scale, rstd, h[i], y[i]);
                *reinterpret_cast<uint4 *>(p.h_out + at + static_cast<size_t>(b) * 8) = pack4(y[i]);
                add_squares(y[i], acc);
            }
        }
    }
    rstd = rstd_of(row_sum<W>(acc.x + acc.y, s_red[1], warp, lane), inv_k, p.eps);

    fp4::let_next_start();
    // n, and for kNv its largest magnitude; a long row's n is formed again for its codes
    uint32_t top = 0, m[P] = {};
    for (int at_c = 0; at_c < (kLong && kOut == fp4::kMx ? 0 : np); at_c += kChunk) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int b = b0 + at_c + i * kStep;
            if (b < np) {
                if (kLong)
                    unpack4(*reinterpret_cast<const uint4 *>(p.h_out + at + static_cast<size_t>(b) * 8), y[i]);
                Pre &f = pre[kAhead ? i : 0];
                if (!kAhead)
                    load_pre(p, int64_t{8} * b, mod, f);
                normalise(f, rstd, y[i], h[i]);
                if constexpr (kOut == kOutBf16)
                    *reinterpret_cast<uint4 *>(p.n_out + at + static_cast<size_t>(b) * 8) = pack4(h[i]);
                else
                    top = max(top, m[i] = fp4::amax8(h[i]));
            }
        }
    }
    if constexpr (kOut != kOutBf16) {
        fp4::Row row{};
        if (kOut == fp4::kNv) {
            row = fp4::row_of(fp4::row_top<W>(top, s_top, warp, lane));
            if (threadIdx.x == 0)
                p.factor[r] = row.factor();
        }
        const int64_t KT = fp4::scale_tiles(p.K, kOut);
        const int np_pad = fp4::pieces_padded<kOut>(KT);
        uint8_t *codes = p.codes + r * (p.K / 2), *scales = p.scales + fp4::scale_row(r, KT);
        for (int at_c = 0; at_c < np_pad; at_c += kChunk) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int b = b0 + at_c + i * kStep;
                if (kLong && b < np) {
                    unpack4(*reinterpret_cast<const uint4 *>(p.h_out + at + static_cast<size_t>(b) * 8), y[i]);
                    load_pre(p, int64_t{8} * b, mod, pre[0]);
                    normalise(pre[0], rstd, y[i], h[i]);
                    m[i] = fp4::amax8(h[i]);
                }
                fp4::store_piece<kOut>(codes, scales, b, b < np, np_pad, row, h[i], m[i]);
            }
        }
    }
}

} // namespace bnorm
} // namespace w8a8
