// fp4_host.cuh -- host side of the 4-bit linear and of the fused block norm: choice of
// variant, tensor maps and launches.  Included by w8a8.cu inside its unnamed namespace,
// after the helpers it shares (device table, pointer checks, make_map).

// ------------------------------------------------------------------ sizes and checks
// Longest row of the 4-bit operators and of the block norm: offsets inside a row, 8 bytes of
// scale tiles a value at the most, stay below 2^32.
constexpr int64_t kMaxRowK = int64_t{1} << 24;

bool fp4_format_ok(int format) { return format == W8A8_FP4_MX || format == W8A8_FP4_NV; }

size_t fp4_scale_bytes(int64_t rows, int64_t K, int format)
{
    return static_cast<size_t>((rows + 127) / 128) * static_cast<size_t>(fp4::scale_tiles(K, format)) * 512;
}

// Quantized matrix in device memory: every buffer present, on this device and aligned.
w8a8_status_t check_fp4(const void *codes, const void *scales, const void *factor, int format)
{
    W8A8_TRY(check_device_ptr(codes));
    W8A8_TRY(check_device_ptr(scales));
    if (format == W8A8_FP4_NV)
        W8A8_TRY(check_device_ptr(factor));
    else if (factor != nullptr)
        return W8A8_ERR_INVALID_ARG;
    if (!aligned16(codes) || !aligned16(scales) || (reinterpret_cast<uintptr_t>(factor) & 3u))
        return W8A8_ERR_ALIGNMENT;
    return W8A8_OK;
}

w8a8_status_t fp4_shape(int64_t rows, int64_t K)
{
    if (rows < 0 || K < 0)
        return W8A8_ERR_INVALID_ARG;
    if (K == 0 || K % 32 || K > kMaxRowK || rows > kMaxTmaCoord)
        return W8A8_ERR_SHAPE;
    return W8A8_OK;
}

// Every kernel of this file is launched as a programmatic dependent: its set-up overlaps the
// end of whatever precedes it on the stream, and it reads and writes nothing before that has
// completed (griddepcontrol.wait).  A chain of small kernels saves about 1 us at each.
template <class... Params, class... Args>
w8a8_status_t launch_dependent(void (*kern)(Params...), int64_t grid, int threads, size_t smem, cudaStream_t stream,
                               int cluster, const Args &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e == cudaSuccess ? launch_status() : cuda_fail(e);
}

// ------------------------------------------------------------------ quantizer
// One row a CTA of W warps, P pieces of 8 values a lane.
template <int kFmt, int W, int P>
w8a8_status_t launch_fp4_rows(const fp4::QParams &p, cudaStream_t stream)
{
    return launch_dependent(fp4::quantize_kernel<kFmt, W, P>, p.rows_pad, W * 32, 0, stream, 1, p);
}

// As many CTAs as fit, each with a ring of rows (2 K kRing bytes, 64 KB at most of 16 warps'
// share of 111) and, used or not, all of its share of the SM: see launch_norm_stream.
template <int kFmt, int W>
w8a8_status_t launch_fp4_stream(const fp4::QParams &p, int dev, cudaStream_t stream)
{
    constexpr int kResident = fp4::kStreamWarps / W;
    const size_t budget = 226 * 1024 / kResident - 1024 - sizeof(fp4::StreamTail<W>);
    const size_t smem = budget + sizeof(fp4::StreamTail<W>);
    auto kern = fp4::quantize_stream_kernel<kFmt, W>;
    bool &attr_set = g_dev[dev].fp4_stream_attr_set[kFmt][W];
    {
        std::lock_guard<std::mutex> lk(g_mu);
        if (!attr_set) {
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       static_cast<int>(smem));
            if (e != cudaSuccess)
                return cuda_fail(e);
            attr_set = true;
        }
    }
    const int64_t grid = std::min<int64_t>(p.rows, static_cast<int64_t>(g_dev[dev].sms) * kResident);
    return launch_dependent(kern, grid, W * 32, smem, stream, 1, p);
}

// The ring from 2 rows a resident CTA on, where a lane has up to 32 values, with about as many
// warps as that takes (8192 x 10240 nvfp4: 38.4 us with 10, 42.9 with 16; 16384 x 5120: 39.1
// with 5, 41.8 with 8; 3, 6 and 7 gain nothing over 4 and 8).  A row on its own is split over
// as many warps as it fills with 8 values a lane, up to 16.
template <int kFmt>
w8a8_status_t launch_fp4_quantize_t(const fp4::QParams &p, int dev, cudaStream_t stream)
{
    const int64_t k = p.K, per_warp = 2 * g_dev[dev].sms * fp4::kStreamWarps;
    const int64_t warps = (k + 1023) / 1024;
    if (warps <= 16 && p.rows >= per_warp / warps) {
        switch (warps) {
        case 1:
            return launch_fp4_stream<kFmt, 1>(p, dev, stream);
        case 2:
            return launch_fp4_stream<kFmt, 2>(p, dev, stream);
        case 3:
        case 4:
            return launch_fp4_stream<kFmt, 4>(p, dev, stream);
        case 5:
            return launch_fp4_stream<kFmt, 5>(p, dev, stream);
        case 6:
        case 7:
        case 8:
            return launch_fp4_stream<kFmt, 8>(p, dev, stream);
        case 9:
        case 10:
            return launch_fp4_stream<kFmt, 10>(p, dev, stream);
        case 11:
        case 12:
            return launch_fp4_stream<kFmt, 12>(p, dev, stream);
        default:
            return launch_fp4_stream<kFmt, 16>(p, dev, stream);
        }
    }
    if (k <= 256)
        return launch_fp4_rows<kFmt, 1, 1>(p, stream);
    if (k <= 512)
        return launch_fp4_rows<kFmt, 2, 1>(p, stream);
    if (k <= 1024)
        return launch_fp4_rows<kFmt, 4, 1>(p, stream);
    if (k <= 2048)
        return launch_fp4_rows<kFmt, 8, 1>(p, stream);
    if (k <= 4096)
        return launch_fp4_rows<kFmt, 16, 1>(p, stream);
    return launch_fp4_rows<kFmt, 16, 4>(p, stream);
}

w8a8_status_t launch_fp4_quantize(const uint16_t *x, int64_t rows, int64_t K, int format, uint8_t *codes,
                                  uint8_t *scales, float *factor, cudaStream_t stream)
{
    int dev;
    W8A8_TRY(current_device(dev));
    fp4::QParams p{};
    p.x = x;
    p.rows = rows;
    p.rows_pad = (rows + 127) / 128 * 128;
    p.K = K;
    p.codes = codes;
    p.scales = scales;
    p.factor = factor;
    return format == W8A8_FP4_MX ? launch_fp4_quantize_t<fp4::kMx>(p, dev, stream)
                                 : launch_fp4_quantize_t<fp4::kNv>(p, dev, stream);
}

// ------------------------------------------------------------------ product
w8a8_status_t fp4_maps(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t K, int format,
                       uint32_t box_rows, CUtensorMap &mc, CUtensorMap &ms)
{
    W8A8_TRY(make_map(mc, codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, rows, K / 2, box_rows, 128,
                      CU_TENSOR_MAP_SWIZZLE_128B));
    // scale tiles of a row of tiles are contiguous: 8-byte units, 64 a tile
    return make_map(ms, scales, CU_TENSOR_MAP_DATA_TYPE_FLOAT64, 8, (rows + 127) / 128,
                    fp4::scale_tiles(K, format) * 64, 1, static_cast<uint32_t>(fp4::scale_tiles_a_slice(format) * 64),
                    CU_TENSOR_MAP_SWIZZLE_NONE);
}

struct Fp4Operand {
    const uint8_t *codes, *scales;
    const float *factor;
};

template <int kFmt, bool kTma>
w8a8_status_t launch_fp4_pair(const Fp4Operand &x, const Fp4Operand &w, fp4::GemmParams p, cudaStream_t stream)
{
    int dev;
    W8A8_TRY(current_device(dev));
    CUtensorMap mx, mxs, mw, mws, my;
    W8A8_TRY(fp4_maps(x.codes, x.scales, p.M, p.K, kFmt, 128, mx, mxs));
    W8A8_TRY(fp4_maps(w.codes, w.scales, p.N, p.K, kFmt, 64, mw, mws));
    my = mx;
    if (kTma)
        W8A8_TRY(make_map(my, p.y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.M, p.N, 32, 64, CU_TENSOR_MAP_SWIZZLE_128B));
    p.num_tm = static_cast<int32_t>((p.M + 255) / 256);
    p.num_tn = static_cast<int32_t>((p.N + 255) / 256);
    if (static_cast<int64_t>(p.num_tm) * p.num_tn >= (int64_t{1} << 30))
        return W8A8_ERR_SHAPE;
    auto kern = fp4::gemm_pair_kernel<kFmt, kTma>;
    constexpr size_t smem = fp4::kPairSmemBytes<kFmt, kTma>;
    static_assert(smem <= 232448, "exceeds the 227 KB of shared memory a CTA may use");
    int pairs;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        int &known = g_dev[dev].fp4_pairs[kFmt * 2 + kTma];
        if (known == 0) {
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       static_cast<int>(smem));
            if (e != cudaSuccess)
                return cuda_fail(e);
            int n = 0;
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute attr;
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = 2;
            attr.val.clusterDim.y = 1;
            attr.val.clusterDim.z = 1;
            cfg.gridDim = dim3(static_cast<unsigned>(g_dev[dev].sms / 2 * 2));
            cfg.blockDim = dim3(fp4::PairEpi<kTma>::kThreads);
            cfg.dynamicSmemBytes = smem;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) {
                cudaGetLastError();
                n = g_dev[dev].sms / 2;
            }
            known = n;
        }
        pairs = known;
    }
    const int tiles = p.num_tm * p.num_tn, tail = tiles % pairs;
    p.num_full = p.num_units = tiles;
    if (kTma && tail > 0 && 2 * tail <= pairs) {
        p.num_full = tiles - tail;
        p.num_units = tiles + tail;
    }
    return launch_dependent(kern, 2 * std::min(pairs, p.num_units), fp4::PairEpi<kTma>::kThreads, smem, stream, 2, mx, mw,
                            mxs, mws, my, p);
}

// xb: BF16 activations to quantize on the way (kQuant), else null.
template <int kFmt, int BT, bool kQuant>
w8a8_status_t launch_fp4_skinny(const Fp4Operand &x, const uint16_t *xb, const Fp4Operand &w, fp4::GemmParams p,
                                cudaStream_t stream)
{
    int dev;
    W8A8_TRY(current_device(dev));
    CUtensorMap mx, mxs, mw, mws;
    W8A8_TRY(fp4_maps(w.codes, w.scales, p.N, p.K, kFmt, 128, mw, mws));
    mx = mw;
    mxs = mws;
    if (!kQuant)
        W8A8_TRY(fp4_maps(x.codes, x.scales, p.M, p.K, kFmt, BT, mx, mxs));
    p.num_tm = static_cast<int32_t>((p.M + BT - 1) / BT);
    p.num_tn = static_cast<int32_t>((p.N + 127) / 128);
    const int64_t tiles = static_cast<int64_t>(p.num_tm) * p.num_tn;
    if (tiles >= (int64_t{1} << 27))
        return W8A8_ERR_SHAPE;
    auto kern = fp4::gemm_skinny_kernel<kFmt, BT, kQuant>;
    constexpr size_t smem = fp4::kSkinnySmemBytes<kFmt, BT>;
    static_assert(smem <= 232448, "exceeds the 227 KB of shared memory a CTA may use");
    int clusters[2];
    constexpr int slot = kFmt * 5 + (kQuant ? 4 : BT == 16 ? 0 : BT == 32 ? 1 : BT == 64 ? 2 : 3);
    {
        std::lock_guard<std::mutex> lk(g_mu);
        if (!g_dev[dev].fp4_skinny_attr_set[slot]) {
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       static_cast<int>(smem));
            if (e != cudaSuccess)
                return cuda_fail(e);
            g_dev[dev].fp4_skinny_attr_set[slot] = true;
        }
        for (int i = 0; i < 2; ++i) {
            int &n = g_dev[dev].fp4_clusters[i];
            const int size = 2 << i;
            if (n == 0) {
                cudaLaunchConfig_t cfg = {};
                cudaLaunchAttribute attr;
                attr.id = cudaLaunchAttributeClusterDimension;
                attr.val.clusterDim.x = static_cast<unsigned>(size);
                attr.val.clusterDim.y = 1;
                attr.val.clusterDim.z = 1;
                cfg.gridDim = dim3(static_cast<unsigned>(g_dev[dev].sms / size * size));
                cfg.blockDim = dim3(fp4::kSkinnyThreads);
                cfg.dynamicSmemBytes = smem;
                cfg.attrs = &attr;
                cfg.numAttrs = 1;
                if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) {
                    cudaGetLastError();
                    n = g_dev[dev].sms / size;
                }
            }
            clusters[i] = n;
        }
    }
    // K is split while the clusters fit on the device all at once, two CTAs a SM, and leave each
    // CTA enough slices: 4 in clusters of up to 4 (1 x 4096 x 4096: 7.7 us unsplit, 6.7, 6.0 in
    // clusters of 2, 4 and 7.4 of 8), 8 in clusters of 8 (1 x 16384 x 3584, 28 tiles: 9.1 us in
    // clusters of 4, 8.4 of 8).  A cluster takes SMs of one group (GPC), whose number its size need
    // not divide, and tiles past those that fit run in a second wave (37 x 16384 x 4608, 36 tiles:
    // 13.7 us in clusters of 4, 20.4 of 8; 37 x 4096 x 9216, 72 tiles: 8.1 us of 2, 14.1 of 4).
    // The occupancy query counts one CTA a SM, 74 clusters of 2 and 33 of 4.  With two CTAs a SM
    // clusters of 8 and 4 take the SMs that those take there: 33 and, three fewer, 71 were seen
    // to run at once (34 and 72 not).
    int splits = 1;
    const int fit[3] = {2 * clusters[0], clusters[0] - 3, clusters[1]};
    for (int i = 0; i < 3 && tiles <= fit[i] && p.slices >= splits * 2 * (splits < 4 ? 4 : 8); ++i)
        splits *= 2;
    return launch_dependent(kern, tiles * splits, fp4::kSkinnyThreads, smem, stream, splits, mx, mw, mxs, mws, xb, p);
}

template <int kFmt>
w8a8_status_t launch_fp4_gemm_t(const Fp4Operand &x, const Fp4Operand &w, const fp4::GemmParams &p, cudaStream_t stream)
{
    if (p.M <= 16)
        return launch_fp4_skinny<kFmt, 16, false>(x, nullptr, w, p, stream);
    if (p.M <= 32)
        return launch_fp4_skinny<kFmt, 32, false>(x, nullptr, w, p, stream);
    if (p.M <= 64)
        return launch_fp4_skinny<kFmt, 64, false>(x, nullptr, w, p, stream);
    // From 65 tokens on pairs of CTAs, which do not split K, unless the output is so small and K
    // so long that there are no more 128 x 128 tiles than slices of K, and few enough tiles for
    // the other kernel to split it: 1000 x 16384 x 8 20.1 -> 10.0 us, 256 x 16384 x 4096 (64
    // tiles, 64 slices) 23.0 -> 20.2; on the other side 300 x 4096 x 1024 (24, 16) 8.9 us with
    // pairs, 10.4 split, 2000 x 8192 x 512 (64, 32) 13.0 and 14.8.  Unsplit it loads twice the
    // operands that the pairs do for a product: 1664 x 65536 x 1408 (143 tiles, 256 slices)
    // 86 us split in two, 92 with pairs, 1664 x 65536 x 1536 (156, 256) 118 unsplit, 89 with pairs.
    int dev;
    W8A8_TRY(current_device(dev));
    const int64_t tiles = ((p.M + 127) / 128) * ((p.N + 127) / 128);
    if (tiles <= p.slices && tiles <= g_dev[dev].sms)
        return launch_fp4_skinny<kFmt, 128, false>(x, nullptr, w, p, stream);
    return p.N % 8 == 0 && aligned16(p.y) ? launch_fp4_pair<kFmt, true>(x, w, p, stream)
                                          : launch_fp4_pair<kFmt, false>(x, w, p, stream);
}

fp4::GemmParams fp4_gemm_params(const Fp4Operand &x, int64_t M, int64_t K, const w8a8_fp4_weight_t *w,
                                const uint16_t *bias, uint16_t *y)
{
    fp4::GemmParams p{};
    p.M = M;
    p.N = w->N;
    p.K = K;
    p.slices = static_cast<int32_t>((K + fp4::kSliceK - 1) / fp4::kSliceK);
    p.xf = x.factor;
    p.wf = w->factor;
    p.bias = bias;
    p.y = y;
    return p;
}

w8a8_status_t launch_fp4_gemm(const Fp4Operand &x, int64_t M, int64_t K, const w8a8_fp4_weight_t *w,
                              const uint16_t *bias, uint16_t *y, cudaStream_t stream)
{
    const fp4::GemmParams p = fp4_gemm_params(x, M, K, w, bias, y);
    const Fp4Operand wo{w->codes, w->scales, w->factor};
    return w->format == W8A8_FP4_MX ? launch_fp4_gemm_t<fp4::kMx>(x, wo, p, stream)
                                    : launch_fp4_gemm_t<fp4::kNv>(x, wo, p, stream);
}

// The linear of at most fp4::kQuantRows rows: quantization and product in one kernel.
w8a8_status_t launch_fp4_linear_few(const uint16_t *x, int64_t M, int64_t K, const w8a8_fp4_weight_t *w,
                                    const uint16_t *bias, uint16_t *y, cudaStream_t stream)
{
    const fp4::GemmParams p = fp4_gemm_params(Fp4Operand{}, M, K, w, bias, y);
    const Fp4Operand wo{w->codes, w->scales, w->factor};
    return w->format == W8A8_FP4_MX
               ? launch_fp4_skinny<fp4::kMx, 16, true>(Fp4Operand{}, x, wo, p, stream)
               : launch_fp4_skinny<fp4::kNv, 16, true>(Fp4Operand{}, x, wo, p, stream);
}

// A weight record: consistent fields; the buffers are checked by whoever uses them.  A weight
// without rows has none (an empty tensor's address may be null).
w8a8_status_t check_fp4_weight(const w8a8_fp4_weight_t *w, int64_t K)
{
    if (w == nullptr || w->N < 0 || w->K != K || !fp4_format_ok(w->format))
        return W8A8_ERR_INVALID_ARG;
    if ((w->codes == nullptr) != (w->scales == nullptr))
        return W8A8_ERR_INVALID_ARG;
    if (w->codes == nullptr && w->w_bf16 == nullptr && K > 0 && w->N > 0)
        return W8A8_ERR_INVALID_ARG;
    return W8A8_OK;
}

// ------------------------------------------------------------------ block norm
template <int kOut, int W, int P, bool kLong>
w8a8_status_t launch_norm_rows(const bnorm::Params &p, cudaStream_t stream)
{
    const int64_t grid = kOut == bnorm::kOutBf16 ? p.M : p.M_pad;
    return launch_dependent(bnorm::row_kernel<kOut, W, P, kLong>, grid, W * 32, 0, stream, 1, p);
}

// As many CTAs as fit, each with a ring of `stages` rows.
template <int kOut, int W, int P>
w8a8_status_t launch_norm_stream(bnorm::Params p, int dev, cudaStream_t stream)
{
    constexpr int kResident = P > 2 ? 1 : bnorm::kStreamWarps / W;    // CTAs a SM
    const size_t budget = 226 * 1024 / kResident - 1024 - sizeof(bnorm::StreamTail<W>);
    // About 64 KB of rows in flight on a SM, at least two rows a CTA (three where it is alone
    // and its rows are no longer than that): 32768 x 4096 169 us with 2 rows of 16 KB on each of
    // two CTAs, 188 with 3, 191 with 6 (as much is written as read, and the reads of a deeper
    // ring crowd the writes); 8192 x 8192, one CTA, 93 us with 2 rows, 88 with 3, 89 with 6.
    const size_t row = 4 * static_cast<size_t>(p.K), want = (64 * 1024 / kResident + row / 2) / row;
    p.stages = static_cast<int32_t>(
        std::min<size_t>({bnorm::kMaxRing, budget / row, std::max<size_t>(want, kResident == 1 && P <= 2 ? 3 : 2)}));
    // P <= 2: all of a CTA's share of the SM, used or not, for with less more CTAs fit on some
    // SMs than the grid has for each (32768 x 1536 nvfp4: 98 us for 87).  P > 2: the factors are
    // read again for each row, and what the ring leaves is L1 that they stay in (4096 x 16384:
    // 108 us, 123 with the whole share).
    const size_t most = budget + sizeof(bnorm::StreamTail<W>);
    const size_t smem = P > 2 ? p.stages * row + sizeof(bnorm::StreamTail<W>) : most;
    auto kern = bnorm::stream_kernel<kOut, W, P>;
    bool &attr_set = g_dev[dev].norm_stream_attr_set[kOut + 1][P > 2 ? 14 + P : W];
    {
        std::lock_guard<std::mutex> lk(g_mu);
        if (!attr_set) {
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       static_cast<int>(most));
            if (e != cudaSuccess)
                return cuda_fail(e);
            attr_set = true;
        }
    }
    const int64_t grid = std::min<int64_t>(p.M, static_cast<int64_t>(g_dev[dev].sms) * kResident);
    return launch_dependent(kern, grid, W * 32, smem, stream, 1, p);
}

// The ring from 4 rows a resident CTA on.  There a lane has 16 values (24 or 32 in rows of
// more than 8192: 8192 x 12288 nvfp4 206 us with 24, 273 with 32), which spreads a row's
// reductions over enough of them, and a row as many warps as that takes, for idle ones are
// places that another row could have: 32768 x 2560 nvfp4 126 us with 5 warps, 176 with 8 (bf16
// 109, 125), 32768 x 1280 75 us with 3, 84 with 4, 16384 x 6144 177 us with 12, 196 with 16; 14
// for 16 loses (16384 x 7168: 208 us, 201).  A row on its own is split over as many warps as it
// fills.
template <int kOut>
w8a8_status_t launch_block_norm(const bnorm::Params &p, cudaStream_t stream)
{
    int dev;
    W8A8_TRY(current_device(dev));
    const int64_t k = p.K, per_warp = 4 * g_dev[dev].sms * bnorm::kStreamWarps;
    const int64_t warps = (k + 511) / 512;
    if (warps <= 32 && p.M >= per_warp / std::min<int64_t>(warps, 16)) {
        switch (warps) {
        case 1:
            return launch_norm_stream<kOut, 1, 2>(p, dev, stream);
        case 2:
            return launch_norm_stream<kOut, 2, 2>(p, dev, stream);
        case 3:
            return launch_norm_stream<kOut, 3, 2>(p, dev, stream);
        case 4:
            return launch_norm_stream<kOut, 4, 2>(p, dev, stream);
        case 5:
            return launch_norm_stream<kOut, 5, 2>(p, dev, stream);
        case 6:
            return launch_norm_stream<kOut, 6, 2>(p, dev, stream);
        case 7:
        case 8:
            return launch_norm_stream<kOut, 8, 2>(p, dev, stream);
        case 9:
        case 10:
            return launch_norm_stream<kOut, 10, 2>(p, dev, stream);
        case 11:
        case 12:
            return launch_norm_stream<kOut, 12, 2>(p, dev, stream);
        case 13:
        case 14:
        case 15:
        case 16:
            return launch_norm_stream<kOut, 16, 2>(p, dev, stream);
        case 17:
        case 18:
        case 19:
        case 20:
        case 21:
        case 22:
        case 23:
        case 24:
            return launch_norm_stream<kOut, 16, 3>(p, dev, stream);
        default:
            return launch_norm_stream<kOut, 16, 4>(p, dev, stream);
        }
    }
    if (k <= 256)
        return launch_norm_rows<kOut, 1, 1, false>(p, stream);
    if (k <= 512)
        return launch_norm_rows<kOut, 2, 1, false>(p, stream);
    if (k <= 1024)
        return launch_norm_rows<kOut, 4, 1, false>(p, stream);
    if (k <= 2048)
        return launch_norm_rows<kOut, 8, 1, false>(p, stream);
    if (k <= 4096)
        return launch_norm_rows<kOut, 16, 1, false>(p, stream);
    if (k <= 8192)
        return launch_norm_rows<kOut, 16, 2, false>(p, stream);
    if (k <= 16384)
        return launch_norm_rows<kOut, 16, 4, false>(p, stream);
    return launch_norm_rows<kOut, 16, 2, true>(p, stream);
}

// Arguments that both forms share -> p.
w8a8_status_t block_norm_common(const uint16_t *h, const uint16_t *y, int post_norm, const uint16_t *post_gamma,
                                const uint16_t *gate, float res_scale, const uint16_t *pre_gamma,
                                const uint16_t *scale, const uint16_t *shift, int64_t T, float eps, int64_t M,
                                int64_t K, uint16_t *h_out, bnorm::Params &p)
{
    if (M < 0 || K < 0 || T <= 0 || !(eps >= 0.0f) || !(eps <= 3.4e38f) || !(res_scale >= -3.4e38f) ||
        !(res_scale <= 3.4e38f) || (post_gamma != nullptr && !post_norm))
        return W8A8_ERR_INVALID_ARG;
    if (K == 0 || K % 8 || M % T || K > kMaxRowK || M > kMaxTmaCoord)
        return W8A8_ERR_SHAPE;
    if (M == 0)
        return W8A8_OK;
    W8A8_TRY(check_device_ptr(h));
    W8A8_TRY(check_device_ptr(y));
    W8A8_TRY(check_device_ptr(h_out));
    const uint16_t *columns[5] = {post_gamma, gate, pre_gamma, scale, shift};
    for (const uint16_t *c : columns) {
        if (c == nullptr)
            continue;
        W8A8_TRY(check_device_ptr(c));
        if (!aligned16(c))
            return W8A8_ERR_ALIGNMENT;
    }
    if (!aligned16(h) || !aligned16(y) || !aligned16(h_out))
        return W8A8_ERR_ALIGNMENT;
    p = bnorm::Params{};
    p.h = h;
    p.y = y;
    p.post_gamma = post_gamma;
    p.pre_gamma = pre_gamma;
    p.gate = gate;
    p.scale = scale;
    p.shift = shift;
    p.M = M;
    p.M_pad = (M + 127) / 128 * 128;
    p.K = K;
    p.T = T;
    p.eps = eps;
    p.res_scale = res_scale;
    p.post_norm = post_norm;
    p.h_out = h_out;
    return W8A8_OK;
}
