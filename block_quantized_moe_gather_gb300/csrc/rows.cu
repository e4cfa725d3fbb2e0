// Activation rows into expert order and back: dispatch, combine and their
// gradients (the public form of the row moves inside the MoE layer).
//
// With inv[t][j] the sorted row of pair (t, j):
//   dispatch           xs[inv[t][j]] = x[t]
//   dispatch backward  dx[t] = sum_j dxs[inv[t][j]]
//   combine            y[t] (+)= sum_j w[t][j] ys[inv[t][j]]
//   combine backward   dys[inv[t][j]] = w[t][j] dy[t],  dw[t][j] = <dy[t], ys[inv[t][j]]>
//
// Every kernel is bound by memory.  Going by token rather than by sorted row
// reads or writes the token's row once instead of k times, and the k sorted
// rows exactly once; no thread shares an output, so there are no atomics and
// every sum has a fixed order.
#include <algorithm>

#include "row_types.cuh"

namespace {

constexpr int kThreads = 256;

// Sorted row of pair f; -1 if it was dropped or is out of range (recorded).
__device__ __forceinline__ int sorted_row(const int32_t* inv, int64_t f, int64_t pairs, int32_t* status) {
    const int r = __ldg(inv + f);
    if (r < -1 || r >= pairs) {
        bq::set_device_error(status, BQ_DEV_BAD_ROW);
        return -1;
    }
    return r;
}

// One 16-byte vector of a token's row to its k sorted rows.
__global__ void __launch_bounds__(kThreads)
dispatch_kernel(const uint8_t* __restrict__ x, int64_t ldx, int T, int vecs, const int32_t* __restrict__ inv, int k,
                uint8_t* __restrict__ xs, int64_t ldxs, int32_t* status) {
    const int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x;
    if (i >= (int64_t)T * vecs) return;
    const int64_t t = i / vecs;
    const int c = (int)(i - t * vecs);
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(x + t * ldx) + c);
    for (int j = 0; j < k; ++j) {
        const int r = sorted_row(inv, t * k + j, (int64_t)T * k, status);
        if (r >= 0) reinterpret_cast<uint4*>(xs + r * ldxs)[c] = v;
    }
}

// One 16-byte vector of y[t].  weights NULL: a plain sum.
template <int DT>
__global__ void __launch_bounds__(kThreads)
combine_rows_kernel(const uint8_t* __restrict__ ys, int64_t ldys, int T, int vecs, const int32_t* __restrict__ inv,
                    const float* __restrict__ weights, int k, int accumulate, uint8_t* __restrict__ y, int64_t ldy,
                    int32_t* status) {
    using V = bq::RowVec<DT>;
    const int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x;
    if (i >= (int64_t)T * vecs) return;
    const int64_t t = i / vecs;
    const int c = (int)(i - t * vecs);
    float acc[V::N];
#pragma unroll
    for (int n = 0; n < V::N; ++n) acc[n] = 0.f;
    for (int j = 0; j < k; ++j) {
        const int r = sorted_row(inv, t * k + j, (int64_t)T * k, status);
        if (r < 0) continue;
        const float w = weights ? __ldg(weights + t * k + j) : 1.f;
        float f[V::N];
        V::unpack(__ldg(reinterpret_cast<const uint4*>(ys + r * ldys) + c), f);
#pragma unroll
        for (int n = 0; n < V::N; ++n) acc[n] = __fmaf_rn(w, f[n], acc[n]);
    }
    uint4* out = reinterpret_cast<uint4*>(y + t * ldy) + c;
    if (accumulate) {
        float f[V::N];
        V::unpack(*out, f);
#pragma unroll
        for (int n = 0; n < V::N; ++n) acc[n] += f[n];
    }
    *out = V::pack(acc);
}

// One CTA per token: its k rows of dys and its k weight gradients.
template <int DT>
__global__ void __launch_bounds__(kThreads)
combine_backward_kernel(const uint8_t* __restrict__ dy, int64_t lddy, const uint8_t* __restrict__ ys, int64_t ldys,
                        int T, int vecs, const int32_t* __restrict__ inv, const float* __restrict__ weights, int k,
                        uint8_t* __restrict__ dys, int64_t lddys, float* __restrict__ dweights, int32_t* status) {
    using V = bq::RowVec<DT>;
    __shared__ float part[kThreads / 32][8];
    const int64_t t = blockIdx.x;
    float dot[8];
    for (int j = 0; j < 8; ++j) dot[j] = 0.f;
    for (int c = threadIdx.x; c < vecs; c += kThreads) {
        float g[V::N];
        V::unpack(__ldg(reinterpret_cast<const uint4*>(dy + t * lddy) + c), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j >= k) break;
            const int r = sorted_row(inv, t * k + j, (int64_t)T * k, status);
            if (r < 0) continue;
            if (dweights) {
                float f[V::N];
                V::unpack(__ldg(reinterpret_cast<const uint4*>(ys + r * ldys) + c), f);
#pragma unroll
                for (int n = 0; n < V::N; ++n) dot[j] = __fmaf_rn(g[n], f[n], dot[j]);
            }
            if (dys) {
                const float w = __ldg(weights + t * k + j);
                float o[V::N];
#pragma unroll
                for (int n = 0; n < V::N; ++n) o[n] = w * g[n];
                reinterpret_cast<uint4*>(dys + r * lddys)[c] = V::pack(o);
            }
        }
    }
    if (!dweights) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int off = 16; off; off >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], off);
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5][j] = dot[j];
    }
    __syncthreads();
    if (threadIdx.x < k) {
        float s = 0.f;
        for (int w = 0; w < kThreads / 32; ++w) s += part[w][threadIdx.x];
        dweights[t * k + threadIdx.x] = s;
    }
}

bq_status check_pairs(const char* name, int32_t dtype, int32_t T, int32_t H, int32_t k) {
    if (bq::dtype_size(dtype) == 0) return bq::fail(BQ_ERR_FORMAT, "%s: unknown element type %d", name, dtype);
    if (T < 0 || H < 1) return bq::fail(BQ_ERR_SHAPE, "%s: T = %d, H = %d", name, T, H);
    if (k < 1 || k > 8) return bq::fail(BQ_ERR_SHAPE, "%s: k = %d outside [1, 8]", name, k);
    if ((int64_t)T * k > (int64_t)INT32_MAX)
        return bq::fail(BQ_ERR_SHAPE, "%s: T * k = %lld pairs exceeds %d", name, (long long)T * k, INT32_MAX);
    return BQ_OK;
}

bq_status check_list(const char* name, const char* what, const void* p) {
    if (!p) return bq::fail(BQ_ERR_NULL, "%s: %s is NULL", name, what);
    if (!bq::aligned(p, 4)) return bq::fail(BQ_ERR_ALIGN, "%s: %s must be 4-byte aligned", name, what);
    return BQ_OK;
}

// CTAs of one thread per 16-byte vector, or an error when there are too many for a grid.
bq_status vector_grid(const char* name, int T, int vecs, unsigned* grid) {
    const int64_t n = ((int64_t)T * vecs + kThreads - 1) / kThreads;
    if (n > INT32_MAX) return bq::fail(BQ_ERR_SHAPE, "%s: T = %d rows of %d vectors are too many", name, T, vecs);
    *grid = (unsigned)n;
    return BQ_OK;
}

bq_status run_combine(const char* name, const void* ys, int32_t dtype, int32_t T, int32_t H, int64_t ldys,
                      const int32_t* inv, const float* weights, int32_t k, int accumulate, void* y, int64_t ldy,
                      cudaStream_t st) {
    const int es = bq::dtype_size(dtype), vecs = H * es / 16;
    unsigned grid;
    bq_status s;
    if ((s = vector_grid(name, T, vecs, &grid)) != BQ_OK || (s = bq::check_arch()) != BQ_OK) return s;
    auto go = [&](auto kernel) {
        kernel<<<grid, kThreads, 0, st>>>(static_cast<const uint8_t*>(ys), ldys * es, T, vecs, inv, weights, k,
                                          accumulate, static_cast<uint8_t*>(y), ldy * es, bq::device_status_ptr());
    };
    if (dtype == BQ_DT_F32) go(combine_rows_kernel<BQ_DT_F32>);
    else if (dtype == BQ_DT_F16) go(combine_rows_kernel<BQ_DT_F16>);
    else go(combine_rows_kernel<BQ_DT_BF16>);
    bq::note_launch();
    return bq::check_launch(name);
}

}  // namespace

extern "C" bq_status bq_moe_dispatch(const void* x, int32_t dtype, int32_t T, int32_t H, int64_t ldx,
                                     const int32_t* inv, int32_t k, void* xs, int64_t ldxs, bq_stream_t stream) {
    const char* name = "bq_moe_dispatch";
    bq_status s = check_pairs(name, dtype, T, H, k);
    if (s != BQ_OK || T == 0) return s;
    const int es = bq::dtype_size(dtype), vecs = (int)((int64_t)H * es / 16);
    unsigned grid;
    if ((s = bq::check_rows(name, "x", x, H, ldx, es)) != BQ_OK ||
        (s = bq::check_rows(name, "xs", xs, H, ldxs, es)) != BQ_OK || (s = check_list(name, "inv", inv)) != BQ_OK ||
        (s = vector_grid(name, T, vecs, &grid)) != BQ_OK || (s = bq::check_arch()) != BQ_OK)
        return s;
    dispatch_kernel<<<grid, kThreads, 0, (cudaStream_t)stream>>>(static_cast<const uint8_t*>(x), ldx * es, T, vecs, inv,
                                                                 k, static_cast<uint8_t*>(xs), ldxs * es,
                                                                 bq::device_status_ptr());
    bq::note_launch();
    return bq::check_launch(name);
}

extern "C" bq_status bq_moe_dispatch_backward(const void* dxs, int32_t dtype, int32_t T, int32_t H, int64_t ldxs,
                                              const int32_t* inv, int32_t k, void* dx, int64_t ldx,
                                              bq_stream_t stream) {
    const char* name = "bq_moe_dispatch_backward";
    bq_status s = check_pairs(name, dtype, T, H, k);
    if (s != BQ_OK || T == 0) return s;
    const int es = bq::dtype_size(dtype);
    if ((s = bq::check_rows(name, "dxs", dxs, H, ldxs, es)) != BQ_OK ||
        (s = bq::check_rows(name, "dx", dx, H, ldx, es)) != BQ_OK || (s = check_list(name, "inv", inv)) != BQ_OK)
        return s;
    return run_combine(name, dxs, dtype, T, H, ldxs, inv, nullptr, k, 0, dx, ldx, (cudaStream_t)stream);
}

extern "C" bq_status bq_moe_combine(const void* ys, int32_t dtype, int32_t T, int32_t H, int64_t ldys,
                                    const int32_t* inv, const float* weights, int32_t k, int32_t accumulate, void* y,
                                    int64_t ldy, bq_stream_t stream) {
    const char* name = "bq_moe_combine";
    bq_status s = check_pairs(name, dtype, T, H, k);
    if (s != BQ_OK) return s;
    if (accumulate != 0 && accumulate != 1)
        return bq::fail(BQ_ERR_SHAPE, "%s: accumulate must be 0 or 1, not %d", name, accumulate);
    if (T == 0) return BQ_OK;
    const int es = bq::dtype_size(dtype);
    if ((s = bq::check_rows(name, "ys", ys, H, ldys, es)) != BQ_OK ||
        (s = bq::check_rows(name, "y", y, H, ldy, es)) != BQ_OK || (s = check_list(name, "inv", inv)) != BQ_OK ||
        (s = check_list(name, "weights", weights)) != BQ_OK)
        return s;
    return run_combine(name, ys, dtype, T, H, ldys, inv, weights, k, accumulate, y, ldy, (cudaStream_t)stream);
}

extern "C" bq_status bq_moe_combine_backward(const void* dy, int64_t lddy, const void* ys, int64_t ldys, int32_t dtype,
                                             int32_t T, int32_t H, const int32_t* inv, const float* weights, int32_t k,
                                             void* dys, int64_t lddys, float* dweights, bq_stream_t stream) {
    const char* name = "bq_moe_combine_backward";
    bq_status s = check_pairs(name, dtype, T, H, k);
    if (s != BQ_OK || T == 0) return s;
    const int es = bq::dtype_size(dtype);
    if (!dys && !dweights) return bq::fail(BQ_ERR_NULL, "%s: dys and dweights are both NULL", name);
    if ((s = bq::check_rows(name, "dy", dy, H, lddy, es)) != BQ_OK || (s = check_list(name, "inv", inv)) != BQ_OK)
        return s;
    if (dys && ((s = bq::check_rows(name, "dys", dys, H, lddys, es)) != BQ_OK ||
                (s = check_list(name, "weights", weights)) != BQ_OK))
        return s;
    if (dweights && ((s = bq::check_rows(name, "ys", ys, H, ldys, es)) != BQ_OK ||
                     (s = check_list(name, "dweights", dweights)) != BQ_OK))
        return s;
    if ((s = bq::check_arch()) != BQ_OK) return s;
    auto go = [&](auto kernel) {
        kernel<<<T, kThreads, 0, (cudaStream_t)stream>>>(
            static_cast<const uint8_t*>(dy), lddy * es, static_cast<const uint8_t*>(ys), ldys * es, T, H * es / 16, inv,
            weights, k, static_cast<uint8_t*>(dys), lddys * es, dweights, bq::device_status_ptr());
    };
    if (dtype == BQ_DT_F32) go(combine_backward_kernel<BQ_DT_F32>);
    else if (dtype == BQ_DT_F16) go(combine_backward_kernel<BQ_DT_F16>);
    else go(combine_backward_kernel<BQ_DT_BF16>);
    bq::note_launch();
    return bq::check_launch(name);
}
