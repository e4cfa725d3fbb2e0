// Entry points of the products of FP8 rows with FP8 weights (mm_fp8.cuh has the
// kernels and what they compute), and the choice of a kernel.
#include "mm_fp8.cuh"

namespace {

using namespace bq::fp8mm;

// ---------------------------------------------------------------- host side
bool encode(CUtensorMap* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
            const uint32_t* box) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), dims, strides, box, ones,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows [rows][k] in boxes of 128 bytes x `box` rows.
bool row_map(CUtensorMap* map, const uint8_t* x, int rows, int k, int box) {
    const uint64_t dims[2] = {(uint64_t)k, (uint64_t)rows}, strides[1] = {(uint64_t)k};
    const uint32_t b[2] = {kBlock, (uint32_t)box};
    return encode(map, x, 2, dims, strides, b);
}

// Weights [E][n][k] in boxes of 128 bytes x 128 rows.
bool weight_map(CUtensorMap* map, const uint8_t* w, int E, int n, int k) {
    const uint64_t dims[3] = {(uint64_t)k, (uint64_t)n, (uint64_t)E}, strides[2] = {(uint64_t)k, (uint64_t)n * k};
    const uint32_t b[3] = {kBlock, 128, 1};
    return encode(map, w, 3, dims, strides, b);
}

// A gate/up weight [E][2][n/2][k] in boxes of `box` gate rows and their up rows.
bool gate_up_map(CUtensorMap* map, const uint8_t* w, int E, int n, int k, int box) {
    const uint64_t h = n / 2;
    const uint64_t dims[4] = {(uint64_t)k, h, 2, (uint64_t)E}, strides[3] = {(uint64_t)k, h * k, (uint64_t)n * k};
    const uint32_t b[4] = {kBlock, (uint32_t)box, 2, 1};
    return encode(map, w, 4, dims, strides, b);
}

template <bool SWIGLU, bool EPI>
cudaError_t launch_lanes(const CUtensorMap& map_w, const CUtensorMap& map_x, const EndArgs& a, int64_t items, int split,
                         cudaStream_t st) {
    // per device: the attribute is a property of the function on the current device
    static std::atomic<bool> attr_set[64];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_set[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(mm_lanes_kernel<SWIGLU, EPI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   LaneSmem::kBytes);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(split > 1 ? items * split : std::min<int64_t>(items, kSms)));
    cfg.blockDim = dim3(kLaneThreads);
    cfg.dynamicSmemBytes = LaneSmem::kBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, mm_lanes_kernel<SWIGLU, EPI>, map_w, map_x, static_cast<const ArgsOf<EPI>&>(a), split);
}

bq_status run_mm(const char* name, const uint8_t* x, const float* xscales, int32_t rows, const int32_t* offsets,
                 int32_t E, const uint8_t* w, const float* wscales, int32_t n, int32_t k, int32_t swiglu, void* y,
                 int32_t ydtype, int64_t ldy, cudaStream_t st, const bq_epilogue* epi = nullptr) {
    const int es = bq::dtype_size(ydtype);
    if (es == 0) return bq::fail(BQ_ERR_FORMAT, "%s: unknown element type %d", name, ydtype);
    if (swiglu != 0 && swiglu != 1) return bq::fail(BQ_ERR_SHAPE, "%s: swiglu must be 0 or 1, not %d", name, swiglu);
    if (rows < 0 || n < 1 || k < 16 || k % 16)
        return bq::fail(BQ_ERR_SHAPE, "%s: %d rows, n = %d, k = %d (k must be a positive multiple of 16)", name, rows,
                        n, k);
    if (rows > kMaxSize || n > kMaxSize || k > kMaxSize)
        return bq::fail(BQ_ERR_SHAPE, "%s: %d rows, n = %d, k = %d: more than %d", name, rows, n, k, kMaxSize);
    if (swiglu && n % 256)
        return bq::fail(BQ_ERR_SHAPE, "%s: a gate/up weight needs n = %d to be a multiple of 256", name, n);
    if (E < 1 || E > kMaxExperts || (int64_t)E * n > (int64_t)INT32_MAX)
        return bq::fail(BQ_ERR_SHAPE, "%s: E = %d outside [1, 1024], or E * n beyond %d", name, E, INT32_MAX);
    if (rows == 0) return BQ_OK;
    if (!x || !xscales || !w || !wscales || !y) return bq::fail(BQ_ERR_NULL, "%s: NULL pointer", name);
    const int cols = swiglu ? n / 2 : n;
    if (ldy < cols)
        return bq::fail(BQ_ERR_SHAPE, "%s: rows of y are %lld elements apart, fewer than their %d", name,
                        (long long)ldy, cols);
    if (!bq::aligned(x, 16) || !bq::aligned(w, 16) || !bq::aligned(xscales, 4) || !bq::aligned(wscales, 4) ||
        !bq::aligned(offsets, 4) || !bq::aligned(y, es))
        return bq::fail(BQ_ERR_ALIGN, "%s: x and w must be 16-byte aligned, scales and offsets 4-byte, y to its element",
                        name);
    if (epi && epi->residual && epi->ldr < cols)
        return bq::fail(BQ_ERR_SHAPE, "%s: rows of the residual are %lld elements apart, fewer than their %d", name,
                        (long long)epi->ldr, cols);
    if (epi && (!bq::aligned(epi->bias, 4) || !bq::aligned(epi->residual, es)))
        return bq::fail(BQ_ERR_ALIGN, "%s: the bias must be 4-byte aligned, the residual to its element", name);
    const int experts = offsets ? std::min(E, rows) : 1;   // that can have rows
    // most row chunks and items there can be, for the grid and (as an int) inside the kernel
    auto chunks_of = [&](int most) { return (int64_t)bq::row_chunks(rows, most) + (offsets ? experts : 0); };
    auto tiles_of = [&](int width) { return (int64_t)(cols + width - 1) / width; };
    // Which kernel.  Weights on the lanes: while its items fit one wave (n = k = 4096: 128 rows 11.3 us against 15.0;
    // 192 rows, two waves, 19.4 against 14.7), and for experts of up to 16 rows on average, where both read every
    // weight once and it reads less beside them (128 experts, gate/up 1536 x 2048: 8 rows 69.1 us against 72.2, 16 rows
    // 71.0 against 73.1, 32 rows 85.2 against 74.9).  There the wide tile is the faster one when K is so short that the
    // narrower tile's more items count (down 2048 x 768: 0.3 rows 12.8 against 13.3, 4 rows 38.2 against 35.6).  The
    // average is all the host knows: with 2048 gate/up rows over 128 experts in Zipf(1.1) shares it takes 77.4 us
    // against 69.9, with all of them at one expert, the worst case, 37.2 against 12.5.
    const int kb = (k + kBlock - 1) / kBlock;
    const int64_t lane_items = chunks_of(kLaneRows) * tiles_of(swiglu ? 64 : 128);
    const bool few_rows = offsets && rows <= 16 * (int64_t)experts && !(kb <= 8 && lane_items > 8 * kSms);
    const bool wide = lane_items > kSms && !few_rows;
    const int64_t chunks = chunks_of(wide ? 128 : kLaneRows);
    const int64_t items = wide ? chunks * tiles_of(swiglu ? 128 : 256) : lane_items;
    if (items > INT32_MAX / 2) return bq::fail(BQ_ERR_SHAPE, "%s: %d rows x %d columns are too many", name, rows, cols);
    bq_status s = bq::check_arch();
    if (s != BQ_OK) return s;
    const bq::WaitProbe probe = bq::wait_probe();
    const Args product{xscales, rows, offsets, E, wscales, n, k, kb, (n + kBlock - 1) / kBlock, cols,
                       y, ydtype, ldy, bq::device_status_ptr(), probe.limit_ns, probe.skip_weight_copies, (int)chunks};
    const EndArgs a{product, epi ? epi->bias : nullptr, epi && !swiglu ? epi->act : BQ_ACT_NONE, epi ? epi->scale : 1.f,
                    epi ? epi->residual : nullptr, epi ? epi->ldr : 0};
    // an end that changes nothing is none
    const bool end = epi && (epi->bias || a.act != BQ_ACT_NONE || epi->scale != 1.f || epi->residual);
    CUtensorMap map_w, map_x;
    const bool mapped = swiglu ? gate_up_map(&map_w, w, E, n, k, wide ? 64 : 16) : weight_map(&map_w, w, E, n, k);
    if (!mapped || !row_map(&map_x, x, rows, k, wide ? 128 : LaneSmem::BOX))
        return bq::fail(BQ_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", name);
    cudaError_t e;
    if (wide) {
        if (!end) e = swiglu ? launch_wide<true, END_NONE, false>(map_w, map_x, a, items, st)
                             : launch_wide<false, END_NONE, false>(map_w, map_x, a, items, st);
        else if (swiglu || a.act == BQ_ACT_NONE || a.act == BQ_ACT_RELU || a.act == BQ_ACT_RELU2)
            e = launch_wide_simple_end(map_w, map_x, a, items, swiglu, st);
        else
            e = launch_wide_activation_end(map_w, map_x, a, items, st);
    } else {
        // K split over a cluster while all clusters are resident at once (this GPU holds 76, 36 and 15 clusters of 2, 4
        // and 8 CTAs of this size) and the blocks saved pay for the cluster's sum, whose cost goes with the rows.
        // n = k = 4096, one row: 10.4 / 7.2 / 5.6 us for 1, 2 and 4, and 12.6 for 8, which takes two waves.  Eight blocks:
        // 32 x 1024 x 1024 4.6 us for 8 and 5.2 for 4, 32 x 4096 x 1024 5.5 for 4 and for 1.  Six, n = 1024: 4.2 for 4
        // and 4.4 for 1 with 8 rows, 5.1 and 4.8 with 32.  A cluster of 2 gains little from many rows: 32 x 8192 6.5 us
        // against 5.6 unsplit at k = 1024, 7.4 against 7.3 at 2048 and 9.4 against 11.0 at 4096; 4 rows 4.8 against 5.1
        // already at 1024.
        const bool few = rows <= 8;
        int split = 1;
        if (items <= 15 && kb >= 8) split = 8;
        else if (items <= 36 && kb >= (few ? 6 : 8)) split = 4;
        else if (items <= 76 && kb >= (few ? 8 : 16)) split = 2;
        if (end) e = swiglu ? launch_lanes<true, true>(map_w, map_x, a, items, split, st)
                            : launch_lanes<false, true>(map_w, map_x, a, items, split, st);
        else e = swiglu ? launch_lanes<true, false>(map_w, map_x, a, items, split, st)
                        : launch_lanes<false, false>(map_w, map_x, a, items, split, st);
    }
    if (e != cudaSuccess) {
        cudaGetLastError();   // reported here
        return bq::fail(BQ_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
    }
    bq::note_launch();
    return bq::check_launch(name);
}

bq_status check_epilogue(const char* name, const bq_epilogue* epi) {
    if (!epi) return bq::fail(BQ_ERR_NULL, "%s: the epilogue is NULL", name);
    if (epi->act < BQ_ACT_NONE || epi->act > BQ_ACT_RELU2)
        return bq::fail(BQ_ERR_SHAPE, "%s: unknown activation %d", name, epi->act);
    return BQ_OK;
}

}  // namespace

extern "C" bq_status bq_mm_fp8_b128(const uint8_t* x, const float* xscales, int32_t m, const uint8_t* w,
                                    const float* wscales, int32_t n, int32_t k, int32_t swiglu, void* y,
                                    int32_t ydtype, int64_t ldy, bq_stream_t stream) {
    return run_mm("bq_mm_fp8_b128", x, xscales, m, nullptr, 1, w, wscales, n, k, swiglu, y, ydtype, ldy,
                  (cudaStream_t)stream);
}

extern "C" bq_status bq_moe_mm_fp8_b128(const uint8_t* x, const float* xscales, int32_t rows, const int32_t* offsets,
                                        int32_t E, const uint8_t* w, const float* wscales, int32_t n, int32_t k,
                                        int32_t swiglu, void* y, int32_t ydtype, int64_t ldy, bq_stream_t stream) {
    if (rows > 0 && !offsets) return bq::fail(BQ_ERR_NULL, "bq_moe_mm_fp8_b128: offsets is NULL");
    return run_mm("bq_moe_mm_fp8_b128", x, xscales, rows, offsets, E, w, wscales, n, k, swiglu, y, ydtype, ldy,
                  (cudaStream_t)stream);
}

extern "C" bq_status bq_mm_fp8_b128_epilogue(const uint8_t* x, const float* xscales, int32_t m, const uint8_t* w,
                                             const float* wscales, int32_t n, int32_t k, const bq_epilogue* epi, void* y,
                                             int32_t ydtype, int64_t ldy, bq_stream_t stream) {
    const bq_status s = check_epilogue("bq_mm_fp8_b128_epilogue", epi);
    if (s != BQ_OK) return s;
    return run_mm("bq_mm_fp8_b128_epilogue", x, xscales, m, nullptr, 1, w, wscales, n, k, epi->act == BQ_ACT_SWIGLU, y,
                  ydtype, ldy, (cudaStream_t)stream, epi);
}

extern "C" bq_status bq_moe_mm_fp8_b128_epilogue(const uint8_t* x, const float* xscales, int32_t rows,
                                                 const int32_t* offsets, int32_t E, const uint8_t* w,
                                                 const float* wscales, int32_t n, int32_t k, const bq_epilogue* epi,
                                                 void* y, int32_t ydtype, int64_t ldy, bq_stream_t stream) {
    const char* name = "bq_moe_mm_fp8_b128_epilogue";
    const bq_status s = check_epilogue(name, epi);
    if (s != BQ_OK) return s;
    if (rows > 0 && !offsets) return bq::fail(BQ_ERR_NULL, "%s: offsets is NULL", name);
    return run_mm(name, x, xscales, rows, offsets, E, w, wscales, n, k, epi->act == BQ_ACT_SWIGLU, y, ydtype, ldy,
                  (cudaStream_t)stream, epi);
}
