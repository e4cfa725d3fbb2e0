// 16-byte vectors of plain rows (bq_dtype) as fp32 values, and host-side
// checks shared by the entry points that take such rows.
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "bq_internal.cuh"

namespace bq {

inline int dtype_size(int dtype) {
    return dtype == BQ_DT_F32 ? 4 : (dtype == BQ_DT_F16 || dtype == BQ_DT_BF16) ? 2 : 0;
}

// A matrix of `rows` rows of `cols` elements, ld elements apart, read or
// written in 16-byte vectors.
inline bq_status check_rows(const char* name, const char* what, const void* p, int cols, int64_t ld, int es) {
    if (!p) return fail(BQ_ERR_NULL, "%s: %s is NULL", name, what);
    if (ld < cols) return fail(BQ_ERR_SHAPE, "%s: rows of %s are %lld elements apart, fewer than their %d elements",
                               name, what, (long long)ld, cols);
    if (!aligned(p, 16) || ((int64_t)cols * es) % 16 || (ld * es) % 16)
        return fail(BQ_ERR_ALIGN, "%s: rows of %s must start and end on 16-byte boundaries", name, what);
    return BQ_OK;
}

// Calls f with k as a compile-time constant (1..8).
template <typename F>
void with_k(int k, F f) {
    switch (k) {
        case 1: f(std::integral_constant<int, 1>()); break;
        case 2: f(std::integral_constant<int, 2>()); break;
        case 3: f(std::integral_constant<int, 3>()); break;
        case 4: f(std::integral_constant<int, 4>()); break;
        case 5: f(std::integral_constant<int, 5>()); break;
        case 6: f(std::integral_constant<int, 6>()); break;
        case 7: f(std::integral_constant<int, 7>()); break;
        default: f(std::integral_constant<int, 8>()); break;
    }
}

// One 16-byte vector of row type DT as N fp32 values.
template <int DT> struct RowVec;

template <> struct RowVec<BQ_DT_F32> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(uint4 v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

template <> struct RowVec<BQ_DT_F16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(uint4 v, float (&f)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = __half22float2(u32_as_h2(w[i]));
            f[2 * i] = p.x; f[2 * i + 1] = p.y;
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = h2_as_u32(__floats2half2_rn(f[2 * i], f[2 * i + 1]));
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <> struct RowVec<BQ_DT_BF16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(uint4 v, float (&f)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // a bf16 is the upper half of its fp32
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// One value rounded to row type `dtype` and stored at element i of y.
__device__ __forceinline__ void store_value(void* y, int64_t i, int dtype, float v) {
    if (dtype == BQ_DT_F32) static_cast<float*>(y)[i] = v;
    else if (dtype == BQ_DT_F16) static_cast<__half*>(y)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(y)[i] = __float2bfloat16_rn(v);
}

}  // namespace bq
