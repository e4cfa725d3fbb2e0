// Shared by the two directions of the residual norm: row types, packed fp32
// arithmetic, sums over a row, argument checks.
#pragma once

#include <algorithm>
#include <atomic>

#include "packed_f32.cuh"
#include "row_types.cuh"

namespace bq {
namespace resnorm {

constexpr int kMaxH = 16384;
constexpr int kSms = 152;
constexpr int kAny = -1;   // a row type that is read from the arguments

enum { GATE_NONE = BQ_GATE_NONE, GATE_TOKEN = BQ_GATE_TOKEN, GATE_CHANNEL = BQ_GATE_CHANNEL, GATE_FULL = BQ_GATE_FULL };

struct Rows {
    uint8_t* p;
    int ld16;      // from row to row, in units of 16 bytes: a product with a row number takes one instruction
    int dtype;

    __device__ __forceinline__ uint8_t* row(int64_t t) const { return p + ((int64_t)(int)t * ld16) * 16; }
};

struct Gate {
    const uint8_t* p;
    int dtype, kind, sigmoid;
};

__host__ __device__ __forceinline__ int vec_bytes(int dtype) { return dtype == BQ_DT_F32 ? 32 : 16; }   // of eight values

// Eight values of a row, in pairs: without the packed instructions these kernels would be bound by issue.
struct Vec {
    f32x2 p[4];
};

__device__ __forceinline__ Vec same8(float v) { return {both(v), both(v), both(v), both(v)}; }

// From their 16 bytes, or the two 16-byte halves of fp32.
template <int DT>
__device__ __forceinline__ Vec unpack8(const uint4& lo, const uint4& hi, int dtype) {
    const int dt = DT == kAny ? dtype : DT;
    Vec r;
    if (dt == BQ_DT_F32) {
        r.p[0] = two(__uint_as_float(lo.x), __uint_as_float(lo.y));
        r.p[1] = two(__uint_as_float(lo.z), __uint_as_float(lo.w));
        r.p[2] = two(__uint_as_float(hi.x), __uint_as_float(hi.y));
        r.p[3] = two(__uint_as_float(hi.z), __uint_as_float(hi.w));
    } else {
        float f[8];
        if (dt == BQ_DT_F16) bq::RowVec<BQ_DT_F16>::unpack(lo, f);
        else bq::RowVec<BQ_DT_BF16>::unpack(lo, f);
#pragma unroll
        for (int j = 0; j < 4; ++j) r.p[j] = two(f[2 * j], f[2 * j + 1]);
    }
    return r;
}

// Vector i of a row in global memory.
template <int DT>
__device__ __forceinline__ Vec load8(const uint8_t* row, int i, int dtype) {
    const bool wide = (DT == kAny ? dtype : DT) == BQ_DT_F32;
    const uint4* p = reinterpret_cast<const uint4*>(row) + (wide ? 2 * i : i);
    const uint4 lo = p[0];
    return unpack8<DT>(lo, wide ? p[1] : lo, dtype);
}

template <int DT>
__device__ __forceinline__ void store8(uint8_t* row, int i, int dtype, const Vec& v) {
    const int dt = DT == kAny ? dtype : DT;
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 x = parts_of(v.p[j]);
        f[2 * j] = x.x;
        f[2 * j + 1] = x.y;
    }
    if (dt == BQ_DT_F32) {
        reinterpret_cast<float4*>(row)[2 * i] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(row)[2 * i + 1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        reinterpret_cast<uint4*>(row)[i] =
            dt == BQ_DT_F16 ? bq::RowVec<BQ_DT_F16>::pack(f) : bq::RowVec<BQ_DT_BF16>::pack(f);
    }
}

// One value, as its bits; and its value.
__device__ __forceinline__ uint32_t load_raw(const uint8_t* p, int64_t i, int dtype) {
    return dtype == BQ_DT_F32 ? reinterpret_cast<const uint32_t*>(p)[i] : reinterpret_cast<const uint16_t*>(p)[i];
}

__device__ __forceinline__ float raw_value(uint32_t raw, int dtype) {
    return dtype == BQ_DT_F32   ? __uint_as_float(raw)
           : dtype == BQ_DT_F16 ? __half2float(__ushort_as_half((unsigned short)raw))
                                : __uint_as_float(raw << 16);
}

__device__ __forceinline__ float load1(const uint8_t* p, int64_t i, int dtype) { return raw_value(load_raw(p, i, dtype), dtype); }

// By the special-function unit's exp2 and reciprocal, off by 2 units in the last place each; the exponent's argument
// adds |v| units to the exponential.
__device__ __forceinline__ float sigmoid_f(float v) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * v));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}

__device__ __forceinline__ Vec sigmoid8(const Vec& v) {
    Vec r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 x = parts_of(v.p[j]);
        r.p[j] = two(sigmoid_f(x.x), sigmoid_f(x.y));
    }
    return r;
}

struct Columns {
    const uint8_t *gain, *post;        // NULL: none
    int gain_dtype;
    Gate gate;
    float scale;
};

// The factor that a row's branch has as a whole: a gate per token, or 1.
__device__ __forceinline__ float token_factor(const Gate& gate, int64_t t, bool live) {
    if (!live || gate.kind != GATE_TOKEN) return 1.f;
    const float f = load1(gate.p, t, gate.dtype);
    return gate.sigmoid ? sigmoid_f(f) : f;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ float peer_load(const float* p, int rank) {
    float v;
    asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %1, %2;\n ld.shared::cluster.f32 %0, [a];\n}\n"
                 : "=f"(v) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return v;
}

// What the sums over a row go through.  Consecutive sums take different halves, so a half is written again only
// behind the barrier of the sum between.
struct SumBuf {
    float warp[2][32][8];
    float cta[2][8];
};

// One sum over the threads of a row, the same in each: lanes and warps (32 at most) by butterflies.
__device__ __forceinline__ float row_sum(float v, SumBuf& buf, int& turn) {
#pragma unroll
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    float (*mine)[8] = buf.warp[turn] + threadIdx.y * warps;
    if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5][0] = v;
    __syncthreads();
    const int w = threadIdx.x & 31;
    v = w < warps ? mine[w][0] : 0.f;
#pragma unroll
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    turn ^= 1;
    return v;
}

// Two sums of 16 warps at most, the same way: a lane holds one of them after the first exchange.
__device__ __forceinline__ void row_sums(float& v0, float& v1, SumBuf& buf, int& turn) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const bool upper = lane & 16;
    float t = (upper ? v1 : v0) + __shfl_xor_sync(0xffffffffu, upper ? v0 : v1, 16);
#pragma unroll
    for (int off = 8; off; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
    if (warps > 1) {
        float (*mine)[8] = buf.warp[turn] + threadIdx.y * warps;
        if ((lane & 15) == 0) mine[threadIdx.x >> 5][lane >> 4] = t;
        __syncthreads();
        t = (lane & 15) < warps ? mine[lane & 15][lane >> 4] : 0.f;
#pragma unroll
        for (int off = 8; off; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
        turn ^= 1;
    }
    v0 = __shfl_sync(0xffffffffu, t, 0);
    v1 = __shfl_sync(0xffffffffu, t, 16);
}

// Eight sums at once, of a row that a cluster's CTAs may share.  Three steps halve the sums that a lane holds while
// they double the lanes added (7 exchanges instead of 24), and the warps' sums are added with a sum a lane.
template <bool CLUSTER>
__device__ __forceinline__ void row_sums(float (&v)[8], SumBuf& buf, int& turn, int ranks) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
    for (int half = 4; half; half >>= 1) {
        const bool upper = lane & (4 * half);
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float send = upper ? v[i] : v[i + half], keep = upper ? v[i + half] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, 4 * half);
        }
    }
    // lanes 4 n .. 4 n + 3 hold sum n
    float t = v[0];
    t += __shfl_xor_sync(0xffffffffu, t, 2);
    t += __shfl_xor_sync(0xffffffffu, t, 1);
    int at = 4;   // lanes that hold different sums
    if (warps > 1 || CLUSTER) {
        float (*mine)[8] = buf.warp[turn] + threadIdx.y * warps;
        if ((lane & 3) == 0) mine[threadIdx.x >> 5][lane >> 2] = t;
        __syncthreads();
        t = 0.f;
        for (int w = lane >> 3; w < warps; w += 4) t += mine[w][lane & 7];
        t += __shfl_xor_sync(0xffffffffu, t, 16);
        t += __shfl_xor_sync(0xffffffffu, t, 8);
        at = 1;
        if (CLUSTER) {
            if (threadIdx.x < 8) buf.cta[turn][threadIdx.x] = t;
            cluster_sync();
            t = 0.f;
            for (int r = 0; r < ranks; ++r) t += peer_load(&buf.cta[turn][lane & 7], r);
        }
        turn ^= 1;
    }
#pragma unroll
    for (int n = 0; n < 8; ++n) v[n] = __shfl_sync(0xffffffffu, t, n * at);
}

// ---------------------------------------------------------------- rows in flight
// Each thread fetches the vectors that it will use itself, rows ahead, into shared memory of its own (cp.async): the
// loads need no registers while they are in flight, and no barrier when they land.
// Where a thread keeps its VPT vectors of a row in flight: planes of 16 bytes per vector of the block (an fp32 vector
// takes two), so that a warp's lie in distinct banks, and places that are constants.
__host__ __device__ constexpr int planes(int dt) { return dt == BQ_DT_F16 || dt == BQ_DT_BF16 ? 1 : 2; }

__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// A thread's vector v of a row into a stage; all of its vectors.
template <int DT, int PLANE, int VPT>
__device__ __forceinline__ void fetch_one(uint32_t dst, const uint8_t* src, int dtype, int v) {
    const bool wide = (DT == kAny ? dtype : DT) == BQ_DT_F32;
    const uint8_t* p = src + v * (int)blockDim.x * (wide ? 32 : 16);
    copy16_async(dst + v * (PLANE / VPT), p);
    if (wide) copy16_async(dst + v * (PLANE / VPT) + PLANE, p + 16);
}

template <int DT, int PLANE, int VPT>
__device__ __forceinline__ void fetch(uint32_t dst, const uint8_t* src, int dtype, const bool (&has)[VPT]) {
#pragma unroll
    for (int v = 0; v < VPT; ++v)
        if (has[v]) fetch_one<DT, PLANE, VPT>(dst, src, dtype, v);
}

template <int DT, int PLANE, int VPT>
__device__ __forceinline__ Vec staged8(const uint8_t* at, int v, int dtype) {
    const uint8_t* p = at + v * (PLANE / VPT);
    const uint4 lo = *reinterpret_cast<const uint4*>(p);
    if ((DT == kAny ? dtype : DT) != BQ_DT_F32) return unpack8<DT>(lo, lo, dtype);
    return unpack8<BQ_DT_F32>(lo, *reinterpret_cast<const uint4*>(p + PLANE), dtype);
}

template <int PLANE, int VPT>
__device__ __forceinline__ void keep8(uint8_t* at, int v, const Vec& x) {
    uint8_t* p = at + v * (PLANE / VPT);
    *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(x.p[0], x.p[1]);
    *reinterpret_cast<ulonglong2*>(p + PLANE) = make_ulonglong2(x.p[2], x.p[3]);
}

template <int PLANE, int VPT>
__device__ __forceinline__ Vec kept8(const uint8_t* at, int v) {
    const uint8_t* p = at + v * (PLANE / VPT);
    const ulonglong2 lo = *reinterpret_cast<const ulonglong2*>(p), hi = *reinterpret_cast<const ulonglong2*>(p + PLANE);
    return {{lo.x, lo.y, hi.x, hi.y}};
}

// Zeros in a thread's places of vectors that it does not have, up to `end` bytes.
template <int PLANE, int VPT>
__device__ __forceinline__ void zero_missing(uint8_t* own, int end, const bool (&has)[VPT]) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        if (has[v]) continue;
        for (int i = v * (PLANE / VPT); i < end; i += PLANE) *reinterpret_cast<uint4*>(own + i) = make_uint4(0, 0, 0, 0);
    }
}

// A thread's column constants as fp32: gain, and scale * post_gain * (a gate per channel), while its first rows are on
// their way.  to_branch NULL: scale alone, which is not kept.
template <int PLANE, bool POST, int VPT>
__device__ __forceinline__ void keep_columns(uint8_t* to_gain, uint8_t* to_branch, const Columns& c, int vec0,
                                             const bool (&has)[VPT]) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        if (!has[v]) continue;
        const int i = vec0 + v * blockDim.x;
        if (c.gain) keep8<PLANE, VPT>(to_gain, v, load8<kAny>(c.gain, i, c.gain_dtype));
        if (!to_branch) continue;
        Vec b = same8(c.scale);
        if (POST) {
            const Vec p = load8<kAny>(c.post, i, c.gain_dtype);
#pragma unroll
            for (int j = 0; j < 4; ++j) b.p[j] = mul2(b.p[j], p.p[j]);
        }
        if (c.gate.kind == GATE_CHANNEL) {
            Vec f = load8<kAny>(c.gate.p, i, c.gate.dtype);
            if (c.gate.sigmoid) f = sigmoid8(f);
#pragma unroll
            for (int j = 0; j < 4; ++j) b.p[j] = mul2(b.p[j], f.p[j]);
        }
        keep8<PLANE, VPT>(to_branch, v, b);
    }
}

// ---------------------------------------------------------------- host side
constexpr size_t kSmemOfSm = 224 * 1024;

// Rows as check_rows, not further apart than Rows can say.
inline bq_status check_matrix(const char* name, const char* what, const void* p, int cols, int64_t ld, int es) {
    const bq_status s = bq::check_rows(name, what, p, cols, ld, es);
    if (s == BQ_OK && ld * es / 16 > INT32_MAX)
        return bq::fail(BQ_ERR_SHAPE, "%s: rows of %s are %lld elements apart", name, what, (long long)ld);
    return s;
}

inline bq_status check_desc(const char* name, const bq_residual_norm_desc* d, bool x) {
    if (!d) return bq::fail(BQ_ERR_NULL, "%s: desc is NULL", name);
    if (d->T < 0 || d->H < 8 || d->H % 8 || d->H > kMaxH)
        return bq::fail(BQ_ERR_SHAPE, "%s: T = %d, H = %d (H must be a multiple of 8, 8 to %d)", name, d->T, d->H, kMaxH);
    const int32_t types[4] = {d->y_dtype, d->h_dtype, x ? d->x_dtype : BQ_DT_F32, d->gain_dtype};
    for (int32_t t : types)
        if (bq::dtype_size(t) == 0) return bq::fail(BQ_ERR_FORMAT, "%s: unknown element type %d", name, t);
    if (d->gate_kind < BQ_GATE_NONE || d->gate_kind > BQ_GATE_FULL)
        return bq::fail(BQ_ERR_SHAPE, "%s: unknown gate kind %d", name, d->gate_kind);
    if (d->gate_sigmoid != 0 && d->gate_sigmoid != 1)
        return bq::fail(BQ_ERR_SHAPE, "%s: gate_sigmoid must be 0 or 1, not %d", name, d->gate_sigmoid);
    const bool gated = d->gate_kind != BQ_GATE_NONE;
    if (gated && bq::dtype_size(d->gate_dtype) == 0)
        return bq::fail(BQ_ERR_FORMAT, "%s: unknown element type %d", name, d->gate_dtype);
    if (!(d->eps >= 0.f) || d->eps > 3.0e38f) return bq::fail(BQ_ERR_SHAPE, "%s: eps must be finite and >= 0", name);
    if (d->T == 0) return BQ_OK;
    if (x && !d->gain) return bq::fail(BQ_ERR_NULL, "%s: gain is NULL", name);
    if (gated && !d->gate) return bq::fail(BQ_ERR_NULL, "%s: gate is NULL", name);
    if (!bq::aligned(d->gain, 16) || !bq::aligned(d->post_gain, 16))
        return bq::fail(BQ_ERR_ALIGN, "%s: gains must be 16-byte aligned", name);
    if (!gated) return BQ_OK;
    const int es = bq::dtype_size(d->gate_dtype);
    if (d->gate_kind == BQ_GATE_FULL) return check_matrix(name, "gate", d->gate, d->H, d->ldgate, es);
    if (!bq::aligned(d->gate, d->gate_kind == BQ_GATE_CHANNEL ? 16 : es))
        return bq::fail(BQ_ERR_ALIGN, "%s: the gate is not aligned", name);
    return BQ_OK;
}

inline Rows rows(const void* p, int64_t ld, int32_t dtype) {
    return {static_cast<uint8_t*>(const_cast<void*>(p)), (int)(ld * bq::dtype_size(dtype) / 16), dtype};
}

inline Columns columns_of(const bq_residual_norm_desc* d, bool x) {
    const Gate gate{static_cast<const uint8_t*>(d->gate), d->gate_dtype, d->gate_kind, d->gate_sigmoid};
    return {x ? static_cast<const uint8_t*>(d->gain) : nullptr, static_cast<const uint8_t*>(d->post_gain), d->gain_dtype,
            gate, d->scale};
}

template <int Y, int H, int X>
struct Types {
    static constexpr int y = Y, h = H, x = X;
};

// Calls f with the row types as constants: one type for all, a 16-bit type with an fp32 block output (as this
// library's MoE layer leaves it) or with an fp32 stream, and a gate per value (if there is one) of y's type; other mixes
// read their types from the arguments.
template <typename F>
void with_types(int y, int h, int x, int gate, F f) {
    constexpr int F32 = BQ_DT_F32, F16 = BQ_DT_F16, BF16 = BQ_DT_BF16;
    if (gate != y) f(Types<kAny, kAny, kAny>());
    else if (y == F32 && h == F32 && x == F32) f(Types<F32, F32, F32>());
    else if (y == F16 && h == F16 && x == F16) f(Types<F16, F16, F16>());
    else if (y == BF16 && h == BF16 && x == BF16) f(Types<BF16, BF16, BF16>());
    else if (y == F32 && h == F16 && x == F16) f(Types<F32, F16, F16>());
    else if (y == F32 && h == BF16 && x == BF16) f(Types<F32, BF16, BF16>());
    else if (y == F16 && h == F32 && x == F16) f(Types<F16, F32, F16>());
    else if (y == BF16 && h == F32 && x == BF16) f(Types<BF16, F32, BF16>());
    else f(Types<kAny, kAny, kAny>());
}

inline bq_status launched(const char* name, cudaError_t e) {
    if (e != cudaSuccess) {
        cudaGetLastError();   // reported here
        return bq::fail(BQ_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
    }
    bq::note_launch();
    return bq::check_launch(name);
}


}  // namespace resnorm
}  // namespace bq
