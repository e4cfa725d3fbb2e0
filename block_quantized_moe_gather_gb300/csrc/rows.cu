// Activation rows into expert order and back: dispatch, combine and their
// gradients (the public form of the row moves inside the MoE layer).
//
// With inv[t][j] the sorted row of pair (t, j):
//   dispatch           xs[inv[t][j]] = x[t]
//   dispatch backward  dx[t] = sum_j dxs[inv[t][j]]
//   combine            y[t] (+)= sum_j w[t][j] ys[inv[t][j]]
//   combine backward   dys[inv[t][j]] = w[t][j] dy[t],  dw[t][j] = <dy[t], ys[inv[t][j]]>
//
// Every kernel is bound by memory (GB300: dispatch 19.3 us, 6.1 TB/s, at 2048
// tokens x 6 rows of 4096 fp16, 13.8 us, 5.5 TB/s, at 2048 x 8 of 2048 bf16; its
// backward pass 19.8 us, 5.9 TB/s, at 2048 x 6 of 4096 bf16; combine 23.7 to
// 26.4 us, 6.4 to 5.7 TB/s, at 2047 x 8 rows of 2048 fp32; its backward pass
// 23.4 us, 6.1 TB/s, at 2048 x 8 rows of 2048 bf16; a decode step's call 1.5 to
// 2 us).  Going by token rather than by sorted row
// reads or writes the token's row once instead of k times, and the k sorted
// rows exactly once; no thread shares an output, so there are no atomics and
// every sum has a fixed order.
#include <algorithm>

#include "row_types.cuh"

namespace {

constexpr int kThreads = 256;

// Sorted row r of a pair, or -1 if it was dropped or is out of range (recorded).
__device__ __forceinline__ int checked_row(int r, int pairs, int32_t* status) {
    if (r < -1 || r >= pairs) {
        bq::set_device_error(status, BQ_DEV_BAD_ROW);
        return -1;
    }
    return r;
}

// The K sorted rows of token t, loaded together.
template <int K>
__device__ __forceinline__ void sorted_rows(const int32_t* inv, int64_t t, int pairs, int32_t* status, int (&r)[K]) {
#pragma unroll
    for (int j = 0; j < K; ++j) r[j] = __ldg(inv + t * K + j);
#pragma unroll
    for (int j = 0; j < K; ++j) r[j] = checked_row(r[j], pairs, status);
}

// Threads of a block: x over the 16-byte vectors of a row, y over tokens.  K is
// a template argument so that the K rows' loads (or stores) are issued
// together: with a loop over k that waits for each row they took 1.3 times as
// long.

// One vector of a token's row to its K sorted rows.
template <int K>
__global__ void __launch_bounds__(kThreads)
dispatch_kernel(const uint8_t* __restrict__ x, int64_t ldx, int T, int vecs, const int32_t* __restrict__ inv,
                uint8_t* __restrict__ xs, int64_t ldxs, int32_t* status) {
    bq::grid_dependency_wait();   // launched behind whatever precedes it on the stream
    bq::allow_dependents();
    const int64_t t = blockIdx.x * (int64_t)blockDim.y + threadIdx.y;
    const int c = blockIdx.y * blockDim.x + threadIdx.x;
    if (t >= T || c >= vecs) return;
    int r[K];
    sorted_rows(inv, t, T * K, status, r);
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(x + t * ldx) + c);
#pragma unroll
    for (int j = 0; j < K; ++j)
        if (r[j] >= 0) reinterpret_cast<uint4*>(xs + r[j] * ldxs)[c] = v;
}

// One vector of y[t].  weights NULL: a plain sum.  Streaming loads and stores: what is read once and written once does
// not push the rest out of the L2 (2047 x 8 rows of 2048 fp32: 27.3 -> 23.6 us).
template <int DT, int K>
__global__ void __launch_bounds__(kThreads)
combine_rows_kernel(const uint8_t* __restrict__ ys, int64_t ldys, int T, int vecs, const int32_t* __restrict__ inv,
                    const float* __restrict__ weights, int accumulate, uint8_t* __restrict__ y, int64_t ldy,
                    int32_t* status) {
    using V = bq::RowVec<DT>;
    bq::grid_dependency_wait();   // launched behind whatever precedes it on the stream
    bq::allow_dependents();
    const int64_t t = blockIdx.x * (int64_t)blockDim.y + threadIdx.y;
    const int c = blockIdx.y * blockDim.x + threadIdx.x;
    if (t >= T || c >= vecs) return;
    int r[K];
    float w[K];
    uint4 raw[K];
    sorted_rows(inv, t, T * K, status, r);
#pragma unroll
    for (int j = 0; j < K; ++j) {
        raw[j] = r[j] >= 0 ? __ldcs(reinterpret_cast<const uint4*>(ys + r[j] * ldys) + c) : make_uint4(0, 0, 0, 0);
        w[j] = weights ? __ldg(weights + t * K + j) : 1.f;
        if (r[j] < 0) w[j] = 0.f;   // 0 * 0 adds nothing, whatever the pair's weight is
    }
    float acc[V::N];
#pragma unroll
    for (int n = 0; n < V::N; ++n) acc[n] = 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j) {
        float f[V::N];
        V::unpack(raw[j], f);
#pragma unroll
        for (int n = 0; n < V::N; ++n) acc[n] = __fmaf_rn(w[j], f[n], acc[n]);
    }
    uint4* out = reinterpret_cast<uint4*>(y + t * ldy) + c;
    if (accumulate) {
        float f[V::N];
        V::unpack(*out, f);
#pragma unroll
        for (int n = 0; n < V::N; ++n) acc[n] += f[n];
    }
    __stcs(out, V::pack(acc));
}

// One CTA per token: its K rows of dys and its K weight gradients.
template <int DT, int K>
__global__ void __launch_bounds__(kThreads)
combine_backward_kernel(const uint8_t* __restrict__ dy, int64_t lddy, const uint8_t* __restrict__ ys, int64_t ldys,
                        int T, int vecs, const int32_t* __restrict__ inv, const float* __restrict__ weights,
                        uint8_t* __restrict__ dys, int64_t lddys, float* __restrict__ dweights, int32_t* status) {
    using V = bq::RowVec<DT>;
    __shared__ float part[kThreads / 32][K];
    bq::grid_dependency_wait();   // launched behind whatever precedes it on the stream
    bq::allow_dependents();
    const int64_t t = blockIdx.x;
    int r[K];
    float w[K], dot[K];
    sorted_rows(inv, t, T * K, status, r);
#pragma unroll
    for (int j = 0; j < K; ++j) {
        w[j] = dys ? __ldg(weights + t * K + j) : 0.f;
        dot[j] = 0.f;
    }
    for (int c = threadIdx.x; c < vecs; c += blockDim.x) {
        uint4 raw[K];
        const uint4 raw_g = __ldg(reinterpret_cast<const uint4*>(dy + t * lddy) + c);
        if (dweights) {
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (r[j] >= 0) raw[j] = __ldg(reinterpret_cast<const uint4*>(ys + r[j] * ldys) + c);
        }
        float g[V::N];
        V::unpack(raw_g, g);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (r[j] < 0) continue;
            if (dys) {
                float o[V::N];
#pragma unroll
                for (int n = 0; n < V::N; ++n) o[n] = w[j] * g[n];
                reinterpret_cast<uint4*>(dys + r[j] * lddys)[c] = V::pack(o);
            }
            if (dweights) {
                float f[V::N];
                V::unpack(raw[j], f);
#pragma unroll
                for (int n = 0; n < V::N; ++n) dot[j] = __fmaf_rn(g[n], f[n], dot[j]);
            }
        }
    }
    if (!dweights) return;
#pragma unroll
    for (int j = 0; j < K; ++j) {
#pragma unroll
        for (int off = 16; off; off >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], off);
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5][j] = dot[j];
    }
    __syncthreads();
    if (threadIdx.x < K) {
        float s = 0.f;
        for (int i = 0; i < (int)blockDim.x / 32; ++i) s += part[i][threadIdx.x];
        dweights[t * K + threadIdx.x] = s;
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

// Blocks of one thread per 16-byte vector of T rows.
struct VectorGrid {
    dim3 grid, block;
};

bq_status vector_grid(const char* name, int T, int vecs, VectorGrid* g) {
    const int x = std::min(kThreads, (vecs + 31) / 32 * 32), y = kThreads / x;
    g->block = dim3(x, y);
    g->grid = dim3(((unsigned)T + y - 1) / y, (vecs + x - 1) / x);
    if (g->grid.y > 65535) return bq::fail(BQ_ERR_SHAPE, "%s: rows of %d vectors are too long", name, vecs);
    return BQ_OK;
}

bq_status run_combine(const char* name, const void* ys, int32_t dtype, int32_t T, int32_t H, int64_t ldys,
                      const int32_t* inv, const float* weights, int32_t k, int accumulate, void* y, int64_t ldy,
                      cudaStream_t st) {
    const int es = bq::dtype_size(dtype), vecs = (int)((int64_t)H * es / 16);
    VectorGrid g;
    bq_status s;
    if ((s = vector_grid(name, T, vecs, &g)) != BQ_OK || (s = bq::check_arch()) != BQ_OK) return s;
    bq::with_k(k, [&](auto kk) {
        constexpr int K = decltype(kk)::value;
        auto go = [&](auto kernel) {
            bq::launch_after(kernel, g.grid, g.block, 0, st, static_cast<const uint8_t*>(ys), ldys * es, T, vecs, inv,
                             weights, accumulate, static_cast<uint8_t*>(y), ldy * es, bq::device_status_ptr());
        };
        if (dtype == BQ_DT_F32) go(combine_rows_kernel<BQ_DT_F32, K>);
        else if (dtype == BQ_DT_F16) go(combine_rows_kernel<BQ_DT_F16, K>);
        else go(combine_rows_kernel<BQ_DT_BF16, K>);
    });
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
    VectorGrid g;
    if ((s = bq::check_rows(name, "x", x, H, ldx, es)) != BQ_OK ||
        (s = bq::check_rows(name, "xs", xs, H, ldxs, es)) != BQ_OK || (s = check_list(name, "inv", inv)) != BQ_OK ||
        (s = vector_grid(name, T, vecs, &g)) != BQ_OK || (s = bq::check_arch()) != BQ_OK)
        return s;
    bq::with_k(k, [&](auto kk) {
        bq::launch_after(dispatch_kernel<decltype(kk)::value>, g.grid, g.block, 0, (cudaStream_t)stream,
                         static_cast<const uint8_t*>(x), ldx * es, T, vecs, inv, static_cast<uint8_t*>(xs), ldxs * es,
                         bq::device_status_ptr());
    });
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
    const int vecs = (int)((int64_t)H * es / 16), threads = std::min(kThreads, (vecs + 31) / 32 * 32);
    bq::with_k(k, [&](auto kk) {
        constexpr int K = decltype(kk)::value;
        auto go = [&](auto kernel) {
            bq::launch_after(kernel, dim3(T), dim3(threads), 0, (cudaStream_t)stream, static_cast<const uint8_t*>(dy),
                             lddy * es, static_cast<const uint8_t*>(ys), ldys * es, T, vecs, inv, weights,
                             static_cast<uint8_t*>(dys), lddys * es, dweights, bq::device_status_ptr());
        };
        if (dtype == BQ_DT_F32) go(combine_backward_kernel<BQ_DT_F32, K>);
        else if (dtype == BQ_DT_F16) go(combine_backward_kernel<BQ_DT_F16, K>);
        else go(combine_backward_kernel<BQ_DT_BF16, K>);
    });
    bq::note_launch();
    return bq::check_launch(name);
}
