// Products of FP8 rows (one scale per 128 values) with FP8 weights (one scale
// per 128 x 128 block), for one weight and for rows sorted by expert.
//
//   y[r][c] = sum_b xs[r][b] ws[c/128][b] * sum_{i in block b} x[r][i] w[c][i]
//
// Simple form: a CTA of 256 threads computes a 64 x 64 tile of y from values
// decoded to fp32 in shared memory; a block's sum is scaled before it joins
// the total.
#include <algorithm>

#include "row_types.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;
constexpr int kBlock = 128;
constexpr int kStep = 32;

struct Args {
    const uint8_t* x;
    const float* xs;
    int rows;
    const int32_t* offsets;   // [E + 1], or NULL: all rows take matrix 0
    int E;
    const uint8_t* w;
    const float* ws;
    int n, k, kb, nb;
    void* y;
    int ydtype;
    int64_t ldy;
    int32_t* status;
};

__device__ __forceinline__ float e4m3_value(uint8_t b) {
    return __low2float(bq::e4m3x2_to_half2(b));
}

// Expert e's rows [lo, hi); none (and the error recorded) where the offsets are not in order.
__device__ void expert_rows(const Args& a, int e, int* lo, int* hi) {
    const int l = __ldg(a.offsets + e), h = __ldg(a.offsets + e + 1);
    const bool ok = 0 <= l && l <= h && h <= a.rows;
    if (!ok) bq::set_device_error(a.status, BQ_DEV_BAD_ROW);
    *lo = ok ? l : 0;
    *hi = ok ? h : 0;
}

template <bool SWIGLU>
__global__ void __launch_bounds__(kThreads) mm_kernel(const Args a) {
    __shared__ float sx[kStep][kTile + 1], sw[SWIGLU ? 2 : 1][kStep][kTile + 1];
    __shared__ int s_where[3];   // expert, first row, end of its rows
    if (threadIdx.x == 0) {
        int e = 0, lo = 0, hi = a.rows, tile = blockIdx.y;
        if (a.offsets) {
            for (; e < a.E; ++e) {
                expert_rows(a, e, &lo, &hi);
                const int tiles = (hi - lo + kTile - 1) / kTile;
                if (tile < tiles) break;
                tile -= tiles;
            }
        }
        s_where[0] = e;
        s_where[1] = lo + tile * kTile;
        s_where[2] = hi;
    }
    __syncthreads();
    const int e = s_where[0], r0 = s_where[1], end = s_where[2];
    if (e >= a.E || r0 >= end) return;
    const int cols = SWIGLU ? a.n / 2 : a.n, c0 = blockIdx.x * kTile;
    const int tr = threadIdx.x / 16, tc = threadIdx.x % 16;
    float total[SWIGLU ? 2 : 1][4][4] = {}, part[SWIGLU ? 2 : 1][4][4] = {};
    for (int k0 = 0; k0 < a.k; k0 += kStep) {
        for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
            const int r = i / kStep, c = i % kStep;
            const bool in_k = k0 + c < a.k;
            sx[c][r] = in_k && r0 + r < end ? e4m3_value(a.x[(int64_t)(r0 + r) * a.k + k0 + c]) : 0.f;
            for (int h = 0; h < (SWIGLU ? 2 : 1); ++h)
                sw[h][c][r] = in_k && c0 + r < cols
                                  ? e4m3_value(a.w[((int64_t)e * a.n + h * cols + c0 + r) * a.k + k0 + c]) : 0.f;
        }
        __syncthreads();
        for (int c = 0; c < kStep; ++c)
            for (int h = 0; h < (SWIGLU ? 2 : 1); ++h)
                for (int i = 0; i < 4; ++i)
                    for (int j = 0; j < 4; ++j)
                        part[h][i][j] = __fmaf_rn(sx[c][tr + 16 * i], sw[h][c][tc + 16 * j], part[h][i][j]);
        __syncthreads();
        if ((k0 + kStep) % kBlock == 0 || k0 + kStep >= a.k) {
            const int b = k0 / kBlock;
            for (int h = 0; h < (SWIGLU ? 2 : 1); ++h)
                for (int i = 0; i < 4; ++i)
                    for (int j = 0; j < 4; ++j) {
                        const int r = r0 + tr + 16 * i, c = c0 + tc + 16 * j;
                        if (r < end && c < cols) {
                            const float s = a.xs[(int64_t)r * a.kb + b] *
                                            a.ws[((int64_t)e * a.nb + (h * cols + c) / kBlock) * a.kb + b];
                            total[h][i][j] = __fmaf_rn(part[h][i][j], s, total[h][i][j]);
                        }
                        part[h][i][j] = 0.f;
                    }
        }
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int r = r0 + tr + 16 * i, c = c0 + tc + 16 * j;
            if (r >= end || c >= cols) continue;
            float v = total[0][i][j];
            if (SWIGLU) v = __fdiv_rn(v, 1.f + expf(-v)) * total[SWIGLU ? 1 : 0][i][j];
            bq::store_value(a.y, (int64_t)r * a.ldy + c, a.ydtype, v);
        }
}

bq_status run_mm(const char* name, const uint8_t* x, const float* xscales, int32_t rows, const int32_t* offsets,
                 int32_t E, const uint8_t* w, const float* wscales, int32_t n, int32_t k, int32_t swiglu, void* y,
                 int32_t ydtype, int64_t ldy, cudaStream_t st) {
    const int es = bq::dtype_size(ydtype);
    if (es == 0) return bq::fail(BQ_ERR_FORMAT, "%s: unknown element type %d", name, ydtype);
    if (swiglu != 0 && swiglu != 1) return bq::fail(BQ_ERR_SHAPE, "%s: swiglu must be 0 or 1, not %d", name, swiglu);
    if (rows < 0 || n < 1 || k < 16 || k % 16)
        return bq::fail(BQ_ERR_SHAPE, "%s: %d rows, n = %d, k = %d (k must be a positive multiple of 16)", name, rows,
                        n, k);
    if (swiglu && n % 256)
        return bq::fail(BQ_ERR_SHAPE, "%s: a gate/up weight needs n = %d to be a multiple of 256", name, n);
    if (E < 1 || E > 1024 || (int64_t)E * n > (int64_t)INT32_MAX)
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
    const int64_t row_tiles = (int64_t)(rows + kTile - 1) / kTile + (offsets ? std::min(E, rows) : 0);
    if (row_tiles > 65535) return bq::fail(BQ_ERR_SHAPE, "%s: %d rows are too many", name, rows);
    bq_status s = bq::check_arch();
    if (s != BQ_OK) return s;
    Args a{x, xscales, rows, offsets, E, w, wscales, n, k, (k + kBlock - 1) / kBlock, (n + kBlock - 1) / kBlock,
           y, ydtype, ldy, bq::device_status_ptr()};
    const dim3 grid((cols + kTile - 1) / kTile, (unsigned)row_tiles);
    if (swiglu) mm_kernel<true><<<grid, kThreads, 0, st>>>(a);
    else mm_kernel<false><<<grid, kThreads, 0, st>>>(a);
    bq::note_launch();
    return bq::check_launch(name);
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
