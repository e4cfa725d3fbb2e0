// Rows quantised to FP8 e4m3 with one fp32 scale per 128 values: alone, and
// on the way into expert order.
//
//   amax = max |v| of the group, scale = max(amax / 448, 2^-126),
//   code = e4m3(448 v / max(amax, 448 2^-126)), half to even, the quotient
//   rounded as if it were exact.
//
// Eight lanes take a group, 16 values each: one 16-byte store of codes per
// lane, and three shuffles for amax.  Bound by memory, with the instructions
// per value close behind (16384 x 768 bf16: 7.4 us, 5.2 TB/s; a sort of 2048 x
// 2048 to 8 experts each 8.0 us, 5.4 TB/s), so maxima are taken two 16-bit
// patterns at a time and a quotient costs one multiply and two integer steps.  |v| is compared as its bit pattern, so
// a NaN (the largest pattern) is found by the same maximum.
//
// Exact codes without a division per value.  r = v * fl(448 / amax) is within
// 2^-22 of the quotient.  For 16-bit values (mantissas V, A < 2^11) the
// quotient 7 V 2^a / A differs from a border B 2^b of two codes (B < 2^5) by
// a relative 1 / (A B) > 2^-16 or not at all; rounding r to 19 bits therefore
// moves it onto the border in the one case and never across it in the other.
// fp32 values can come closer: where r (1 +- 2^-21) round to different codes,
// the quotient is formed again in 64 bits (exact enough: a border is missed
// by 2^-29 or not at all) and rounded to odd on its way to fp32.
// A group with a NaN or an infinity (rare) is coded apart.
#include "row_types.cuh"

namespace {

constexpr int kThreads = 128;
constexpr int kGroup = 128;       // values per scale
constexpr int kPerLane = 16;      // values per lane
constexpr int kLanes = kGroup / kPerLane;
constexpr float kMinScale = 1.17549435e-38f;   // 2^-126

// Codes of (lo, hi) in the low and high byte.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// r, finite, rounded to 19 significant bits.
__device__ __forceinline__ float round19(float r) {
    return __uint_as_float((__float_as_uint(r) + 0x10u) & ~0x1Fu);
}

// 448 v / amax for an e4m3 rounding: truncated to fp32, the last bit set where that lost anything.
__device__ __noinline__ float quotient_to_odd(float v, float amax) {
    const double q = (double)v * 448.0 / (double)amax;
    const float f = __double2float_rz(q);
    return (double)f == q ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// The largest |v| of a vector, as bits of DT's fp32 value.
template <int DT>
__device__ __forceinline__ uint32_t top_bits(uint4 v) {
    if (DT == BQ_DT_F32) {
        return max(max(v.x & 0x7FFFFFFFu, v.y & 0x7FFFFFFFu), max(v.z & 0x7FFFFFFFu, v.w & 0x7FFFFFFFu));
    } else {   // two 16-bit patterns at a time; the result stays packed
        return __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
    }
}

// Codes of the 16 values of a lane in `raw` (zeros past the row's end); returns the group's scale.
template <int DT>
__device__ __forceinline__ float quantise16(const uint4 (&raw)[kPerLane / bq::RowVec<DT>::N], uint32_t (&codes)[4]) {
    using V = bq::RowVec<DT>;
    constexpr int kVecs = kPerLane / V::N;
    float amax;
    if (DT == BQ_DT_F32) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) top = max(top, top_bits<DT>(raw[i]));
#pragma unroll
        for (int off = kLanes / 2; off; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
        amax = __uint_as_float(top);
    } else {
        uint32_t top = __vmaxu2(top_bits<DT>(raw[0]), top_bits<DT>(raw[kVecs - 1]));
#pragma unroll
        for (int off = kLanes / 2; off; off >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, off));
        top = max(top & 0xFFFFu, top >> 16);
        amax = DT == BQ_DT_F16 ? __half2float(__ushort_as_half((unsigned short)top)) : __uint_as_float(top << 16);
    }
    float scale = __fdiv_rn(amax, 448.f);
    if (scale < kMinScale) scale = kMinScale;                    // a NaN stays
    const bool finite = amax <= 3.4028235e38f;
    if (amax < 448.f * kMinScale) amax = 448.f * kMinScale;
    const float inv = __fdiv_rn(448.f, amax);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        float v[V::N];
        V::unpack(raw[i], v);
#pragma unroll
        for (int n = 0; n < V::N; n += 4) {
            uint32_t pair[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float a = v[n + 2 * h], b = v[n + 2 * h + 1];
                const float ra = __fmul_rn(a, inv), rb = __fmul_rn(b, inv);
                if (DT != BQ_DT_F32) {
                    pair[h] = e4m3_pair(round19(ra), round19(rb));
                } else {
                    constexpr float kUp = 1.f + 0x1p-21f, kDown = 1.f - 0x1p-21f;
                    pair[h] = e4m3_pair(ra * kDown, rb * kDown);
                    if (pair[h] != e4m3_pair(ra * kUp, rb * kUp))
                        pair[h] = e4m3_pair(quotient_to_odd(a, amax), quotient_to_odd(b, amax));
                }
                if (!finite) pair[h] = e4m3_pair(ra, rb);   // 0 or NaN
            }
            codes[(i * V::N + n) / 4] = pair[0] | (pair[1] << 16);
        }
    }
    return scale;
}

// The 16 values from `first` on of a row (zeros past its end).
template <int DT>
__device__ __forceinline__ void load16(const uint8_t* row, int first, int k, uint4 (&raw)[kPerLane / bq::RowVec<DT>::N]) {
    constexpr int kVecs = kPerLane / bq::RowVec<DT>::N;
    const uint4* src = reinterpret_cast<const uint4*>(row) + first / bq::RowVec<DT>::N;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) raw[i] = first < k ? __ldcs(src + i) : make_uint4(0, 0, 0, 0);
}

// Groups (row, b) in row-major order, eight lanes each.  K = 0: row r of x to
// row r of q; else token t to its K sorted rows.
template <int DT, int K>
__global__ void __launch_bounds__(kThreads)
quant_kernel(const uint8_t* __restrict__ x, int64_t ldx, int rows, int k, int kb, const int32_t* __restrict__ n_rows,
             const int32_t* __restrict__ inv, uint8_t* __restrict__ q, float* __restrict__ scales, int32_t* status) {
    bq::grid_dependency_wait();   // launched behind whatever precedes it on the stream
    bq::allow_dependents();
    const int limit = n_rows ? min(__ldg(n_rows), rows) : rows;
    const uint32_t g = (uint32_t)((blockIdx.x * (uint64_t)kThreads + threadIdx.x) / kLanes);   // < 2^31
    const uint32_t row = g / (uint32_t)kb;
    const int b = (int)(g - row * kb), part = threadIdx.x % kLanes, first = b * kGroup + part * kPerLane;
    const bool live = (int)row < limit;
    int r[K > 0 ? K : 1];
    r[0] = (int)row;
    if (K > 0) {
#pragma unroll
        for (int j = 0; j < K; ++j) r[j] = live ? __ldg(inv + (int64_t)row * K + j) : -1;
    }
    uint4 raw[kPerLane / bq::RowVec<DT>::N];
    load16<DT>(x + (int64_t)(live ? row : 0) * ldx, live ? first : k, k, raw);
    uint32_t codes[4];
    const float scale = quantise16<DT>(raw, codes);
    if (!live) return;
#pragma unroll
    for (int j = 0; j < (K > 0 ? K : 1); ++j) {
        if (K > 0 && (r[j] < 0 || r[j] >= rows * K)) {
            if (r[j] != -1) bq::set_device_error(status, BQ_DEV_BAD_ROW);
            continue;
        }
        if (first < k) *reinterpret_cast<uint4*>(q + (int64_t)r[j] * k + first) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
        if (part == 0) scales[(int64_t)r[j] * kb + b] = scale;
    }
}

bq_status run_quant(const char* name, const void* x, int32_t dtype, int32_t rows, int32_t k, int64_t ldx,
                    const int32_t* n_rows, const int32_t* inv, int32_t topk, uint8_t* q, float* scales,
                    bq_stream_t stream) {
    const int es = bq::dtype_size(dtype);
    if (es == 0) return bq::fail(BQ_ERR_FORMAT, "%s: unknown element type %d", name, dtype);
    if (rows < 0 || k < 16 || k % 16)
        return bq::fail(BQ_ERR_SHAPE, "%s: %d rows of %d values (a multiple of 16 is needed)", name, rows, k);
    if (topk < 1 || topk > 8) return bq::fail(BQ_ERR_SHAPE, "%s: k = %d outside [1, 8]", name, topk);
    if ((int64_t)rows * topk > (int64_t)INT32_MAX)
        return bq::fail(BQ_ERR_SHAPE, "%s: T * k = %lld pairs exceeds %d", name, (long long)rows * topk, INT32_MAX);
    if (rows == 0) return BQ_OK;
    bq_status s = bq::check_rows(name, "x", x, k, ldx, es);
    if (s != BQ_OK) return s;
    if (!q || !scales) return bq::fail(BQ_ERR_NULL, "%s: q or scales is NULL", name);
    if (!bq::aligned(q, 16) || !bq::aligned(scales, 4) || !bq::aligned(n_rows, 4) || !bq::aligned(inv, 4))
        return bq::fail(BQ_ERR_ALIGN, "%s: q must be 16-byte aligned, scales, n_rows and inv 4-byte", name);
    const int kb = (int)(((int64_t)k + kGroup - 1) / kGroup);   // k may be within a group of 2^31
    if ((int64_t)rows * kb > (int64_t)INT32_MAX)
        return bq::fail(BQ_ERR_SHAPE, "%s: %d rows of %d groups are too many", name, rows, kb);
    const unsigned grid = (unsigned)(((int64_t)rows * kb * kLanes + kThreads - 1) / kThreads);
    if ((s = bq::check_arch()) != BQ_OK) return s;
    auto go = [&](auto kernel) {
        bq::launch_after(kernel, dim3(grid), dim3(kThreads), 0, (cudaStream_t)stream, static_cast<const uint8_t*>(x),
                         ldx * es, rows, k, kb, n_rows, inv, q, scales, bq::device_status_ptr());
    };
    auto go_k = [&](auto kk) {
        constexpr int K = decltype(kk)::value;
        if (dtype == BQ_DT_F32) go(quant_kernel<BQ_DT_F32, K>);
        else if (dtype == BQ_DT_F16) go(quant_kernel<BQ_DT_F16, K>);
        else go(quant_kernel<BQ_DT_BF16, K>);
    };
    if (inv) bq::with_k(topk, go_k);
    else go_k(std::integral_constant<int, 0>());
    bq::note_launch();
    return bq::check_launch(name);
}

}  // namespace

extern "C" bq_status bq_quant_fp8_b128(const void* x, int32_t dtype, int32_t rows, int32_t k, int64_t ldx,
                                       const int32_t* n_rows, uint8_t* q, float* scales, bq_stream_t stream) {
    return run_quant("bq_quant_fp8_b128", x, dtype, rows, k, ldx, n_rows, nullptr, 1, q, scales, stream);
}

extern "C" bq_status bq_moe_dispatch_fp8_b128(const void* x, int32_t dtype, int32_t T, int32_t H, int64_t ldx,
                                              const int32_t* inv, int32_t k, uint8_t* q, float* scales,
                                              bq_stream_t stream) {
    if (T > 0 && !inv) return bq::fail(BQ_ERR_NULL, "bq_moe_dispatch_fp8_b128: inv is NULL");
    return run_quant("bq_moe_dispatch_fp8_b128", x, dtype, T, H, ldx, nullptr, inv, k, q, scales, stream);
}
