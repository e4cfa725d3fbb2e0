// The way out of a block and into the next: the block's output, normalised if
// the block has a norm behind it, gated and scaled, is added to the residual
// stream, and the stream is normalised for the next block, in one pass; and
// the gradients of that pass.
//
//   n(v) = v / sqrt(mean(v^2) + eps),  g = gate, sigmoid(gate) or 1
//   b = post_gain n(y), or y;   h' = residual_scale h + scale g b;   x = gain n(h')
// Backward, with r = 1 / rms(h') and s = 1 / rms(y) (both with eps):
//   G = dh' + r gain dx - h' r^3 mean(gain dx h'),   dgain = sum_t dx h' r
//   dh = residual_scale G,   D = scale G,   dgate = D b (times g (1 - g) under a sigmoid)
//   dpost = sum_t D g y s,   dy = s post D g - y s^3 mean(post D g y), or D g without a post norm
#include <algorithm>

#include "row_types.cuh"

namespace {

constexpr int kMaxH = 16384;
constexpr int kSms = 152;
constexpr int kAny = -1;   // a row type that is read from the arguments

enum { GATE_NONE = BQ_GATE_NONE, GATE_TOKEN = BQ_GATE_TOKEN, GATE_CHANNEL = BQ_GATE_CHANNEL, GATE_FULL = BQ_GATE_FULL };

struct Rows {
    uint8_t* p;
    int64_t ld;    // bytes
    int dtype;
};

struct Gate {
    const uint8_t* p;
    int64_t ld;    // bytes, of a gate per value
    int dtype, kind, sigmoid;
};

// Eight values (a vector of either 16 or 32 bytes) as fp32.
template <int DT>
__device__ __forceinline__ void load8(const uint8_t* row, int i, int dtype, float (&f)[8]) {
    const int dt = DT == kAny ? dtype : DT;
    if (dt == BQ_DT_F32) {
        const float4 a = reinterpret_cast<const float4*>(row)[2 * i], b = reinterpret_cast<const float4*>(row)[2 * i + 1];
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        const uint4 v = reinterpret_cast<const uint4*>(row)[i];
        if (dt == BQ_DT_F16) bq::RowVec<BQ_DT_F16>::unpack(v, f);
        else bq::RowVec<BQ_DT_BF16>::unpack(v, f);
    }
}

template <int DT>
__device__ __forceinline__ void store8(uint8_t* row, int i, int dtype, const float (&f)[8]) {
    const int dt = DT == kAny ? dtype : DT;
    if (dt == BQ_DT_F32) {
        reinterpret_cast<float4*>(row)[2 * i] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(row)[2 * i + 1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        reinterpret_cast<uint4*>(row)[i] =
            dt == BQ_DT_F16 ? bq::RowVec<BQ_DT_F16>::pack(f) : bq::RowVec<BQ_DT_BF16>::pack(f);
    }
}

__device__ __forceinline__ float load1(const uint8_t* p, int64_t i, int dtype) {
    if (dtype == BQ_DT_F32) return reinterpret_cast<const float*>(p)[i];
    if (dtype == BQ_DT_F16) return __half2float(reinterpret_cast<const __half*>(p)[i]);
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}

__device__ __forceinline__ float sigmoid_f(float v) { return 1.f / (1.f + expf(-v)); }

// N sums over the threads of a row (blockDim.x of them), the same in each: lanes by a butterfly, warps in order.
// `buf`: shared [rows of the block][warps of a row][N]; consecutive calls take different ones.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* buf) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int off = 16; off; off >>= 1) v[n] += __shfl_xor_sync(0xffffffffu, v[n], off);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return;
    float* mine = buf + threadIdx.y * warps * N;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int n = 0; n < N; ++n) mine[(threadIdx.x >> 5) * N + n] = v[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = 0.f;
    for (int w = 0; w < warps; ++w)
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] += mine[w * N + n];
}

// ---------------------------------------------------------------- forward
struct ForwardArgs {
    int T, H;
    Rows y, h, out, x;              // x.p NULL: not computed
    const uint8_t *gain, *post;     // post NULL: no norm behind the block
    int gain_dtype;
    Gate gate;
    float scale, residual_scale, eps;
};

constexpr int kForwardThreads = 512;

// blockDim.x threads take a row, a thread the vectors x, x + blockDim.x, ... of it; blockDim.y rows a CTA.
template <int DY, int DH, int DX, int VPT>
__global__ void __launch_bounds__(kForwardThreads)
residual_norm_kernel(const ForwardArgs a) {
    __shared__ float s_buf[2][kForwardThreads / 32];
    bq::grid_dependency_wait();   // launched behind whatever precedes it on the stream
    bq::allow_dependents();
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = t < a.T;
    const int vecs = a.H / 8;
    const uint8_t *y = a.y.p + t * a.y.ld, *h = a.h.p + t * a.h.ld;
    float b[VPT][8], r[VPT][8];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int i = threadIdx.x + v * blockDim.x;
#pragma unroll
        for (int j = 0; j < 8; ++j) b[v][j] = r[v][j] = 0.f;
        if (live && i < vecs) {
            load8<DY>(y, i, a.y.dtype, b[v]);
            load8<DH>(h, i, a.h.dtype, r[v]);
        }
    }
    float norm = 1.f;
    if (a.post) {
        float sum[1] = {0.f};
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[0] = __fmaf_rn(b[v][j], b[v][j], sum[0]);
        row_sums(sum, s_buf[0]);
        norm = rsqrtf(sum[0] / (float)a.H + a.eps);
    }
    float token = 1.f;
    if (live && a.gate.kind == GATE_TOKEN) {
        token = load1(a.gate.p, t, a.gate.dtype);
        if (a.gate.sigmoid) token = sigmoid_f(token);
    }
    float sum[1] = {0.f};
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int i = threadIdx.x + v * blockDim.x;
        if (!live || i >= vecs) continue;
        if (a.post) {
            float p[8];
            load8<kAny>(a.post, i, a.gain_dtype, p);
#pragma unroll
            for (int j = 0; j < 8; ++j) b[v][j] *= norm * p[j];
        }
        if (a.gate.kind >= GATE_CHANNEL) {
            float g[8];
            load8<kAny>(a.gate.kind == GATE_FULL ? a.gate.p + t * a.gate.ld : a.gate.p, i, a.gate.dtype, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) b[v][j] *= a.gate.sigmoid ? sigmoid_f(g[j]) : g[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            r[v][j] = __fmaf_rn(a.scale * token, b[v][j], a.residual_scale * r[v][j]);
            sum[0] = __fmaf_rn(r[v][j], r[v][j], sum[0]);
        }
        store8<DH>(a.out.p + t * a.out.ld, i, a.out.dtype, r[v]);
    }
    if (!a.x.p) return;
    row_sums(sum, s_buf[1]);
    norm = rsqrtf(sum[0] / (float)a.H + a.eps);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int i = threadIdx.x + v * blockDim.x;
        if (!live || i >= vecs) continue;
        float g[8];
        load8<kAny>(a.gain, i, a.gain_dtype, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[v][j] *= norm * g[j];
        store8<DX>(a.x.p + t * a.x.ld, i, a.x.dtype, r[v]);
    }
}

// ---------------------------------------------------------------- backward
struct BackwardArgs {
    int T, H;
    Rows y, out, dout, dx;          // dout.p or dx.p NULL: no gradient comes that way
    Rows dy, dh;
    const uint8_t *gain, *post;
    int gain_dtype;
    Gate gate;
    Rows dgate;                     // of a gate per token (fp32) or per value; p NULL: not computed
    float scale, residual_scale, eps;
    float* part;                    // [arrays][parts][H] column sums: dgain, dpost, dgate per channel
    int sum_gain, sum_post, sum_gate;   // which array each is, or -1
};

constexpr int kBackwardThreads = 256;

// CTAs walk over the rows; a thread's columns stay the same, so it adds their column sums in registers.
template <int DY, int DH, int DX, int VPT>
__global__ void __launch_bounds__(kBackwardThreads)
residual_norm_backward_kernel(const BackwardArgs a) {
    __shared__ float s_buf[2][kBackwardThreads / 32 * 3];
    bq::grid_dependency_wait();   // launched behind whatever precedes it on the stream
    bq::allow_dependents();
    const int vecs = a.H / 8;
    float sums[3][VPT][8];
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) sums[k][v][j] = 0.f;
    const float inv_h = 1.f / (float)a.H;
    for (int64_t t0 = (int64_t)blockIdx.x * blockDim.y; t0 < a.T; t0 += (int64_t)gridDim.x * blockDim.y) {
        const int64_t t = t0 + threadIdx.y;
        const bool live = t < a.T;
        float y[VPT][8], h[VPT][8], d[VPT][8], G[VPT][8];
        float s3[3] = {0.f, 0.f, 0.f};   // h'^2, gain dx h', y^2
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int i = threadIdx.x + v * blockDim.x;
#pragma unroll
            for (int j = 0; j < 8; ++j) y[v][j] = h[v][j] = d[v][j] = G[v][j] = 0.f;
            if (!live || i >= vecs) continue;
            load8<DY>(a.y.p + t * a.y.ld, i, a.y.dtype, y[v]);
            if (a.dout.p) load8<DH>(a.dout.p + t * a.dout.ld, i, a.dout.dtype, G[v]);
            if (a.dx.p) {
                load8<DH>(a.out.p + t * a.out.ld, i, a.out.dtype, h[v]);
                load8<DX>(a.dx.p + t * a.dx.ld, i, a.dx.dtype, d[v]);
                float g[8];
                load8<kAny>(a.gain, i, a.gain_dtype, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    s3[0] = __fmaf_rn(h[v][j], h[v][j], s3[0]);
                    s3[1] = __fmaf_rn(d[v][j] * g[j], h[v][j], s3[1]);
                }
            }
            if (a.post) {
#pragma unroll
                for (int j = 0; j < 8; ++j) s3[2] = __fmaf_rn(y[v][j], y[v][j], s3[2]);
            }
        }
        row_sums(s3, s_buf[0]);
        const float r = rsqrtf(s3[0] * inv_h + a.eps), c = r * r * r * (s3[1] * inv_h);
        const float s = rsqrtf(s3[2] * inv_h + a.eps);
        float token = 1.f;
        if (live && a.gate.kind == GATE_TOKEN) {
            token = load1(a.gate.p, t, a.gate.dtype);
            if (a.gate.sigmoid) token = sigmoid_f(token);
        }
        float s2[2] = {0.f, 0.f};        // post D g y, D b
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int i = threadIdx.x + v * blockDim.x;
            if (!live || i >= vecs) continue;
            if (a.dx.p) {
                float g[8];
                load8<kAny>(a.gain, i, a.gain_dtype, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sums[0][v][j] = __fmaf_rn(d[v][j] * r, h[v][j], sums[0][v][j]);
                    G[v][j] += r * (g[j] * d[v][j]) - h[v][j] * c;
                }
            }
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = a.residual_scale * G[v][j];
            store8<DH>(a.dh.p + t * a.dh.ld, i, a.dh.dtype, o);
            float p[8], b[8];
            if (a.post) {
                load8<kAny>(a.post, i, a.gain_dtype, p);
#pragma unroll
                for (int j = 0; j < 8; ++j) b[j] = y[v][j] * s * p[j];
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) b[j] = y[v][j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) G[v][j] *= a.scale;   // D
            if (a.gate.kind == GATE_TOKEN) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    s2[1] = __fmaf_rn(G[v][j], b[j], s2[1]);
                    G[v][j] *= token;
                }
            } else if (a.gate.kind != GATE_NONE) {
                float g[8], dg[8];
                load8<kAny>(a.gate.kind == GATE_FULL ? a.gate.p + t * a.gate.ld : a.gate.p, i, a.gate.dtype, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    dg[j] = G[v][j] * b[j];
                    if (a.gate.sigmoid) {
                        g[j] = sigmoid_f(g[j]);
                        dg[j] *= g[j] * (1.f - g[j]);
                    }
                    G[v][j] *= g[j];
                }
                if (a.gate.kind == GATE_CHANNEL) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) sums[2][v][j] += dg[j];
                } else if (a.dgate.p) {
                    store8<kAny>(a.dgate.p + t * a.dgate.ld, i, a.dgate.dtype, dg);
                }
            }
            if (a.post) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sums[1][v][j] = __fmaf_rn(G[v][j] * s, y[v][j], sums[1][v][j]);
                    G[v][j] *= p[j];
                    s2[0] = __fmaf_rn(G[v][j], y[v][j], s2[0]);
                }
            } else {
                store8<DY>(a.dy.p + t * a.dy.ld, i, a.dy.dtype, G[v]);
            }
        }
        if (a.post || a.gate.kind == GATE_TOKEN) {
            row_sums(s2, s_buf[1]);
            if (a.gate.kind == GATE_TOKEN && a.dgate.p && live && threadIdx.x == 0)
                reinterpret_cast<float*>(a.dgate.p)[t] = a.gate.sigmoid ? s2[1] * token * (1.f - token) : s2[1];
            if (a.post) {
                const float cy = s * s * s * (s2[0] * inv_h);
#pragma unroll
                for (int v = 0; v < VPT; ++v) {
                    const int i = threadIdx.x + v * blockDim.x;
                    if (!live || i >= vecs) continue;
                    float o[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = s * G[v][j] - y[v][j] * cy;
                    store8<DY>(a.dy.p + t * a.dy.ld, i, a.dy.dtype, o);
                }
            }
        } else if (blockDim.x > 32) {
            __syncthreads();   // s_buf[0] is written again
        }
    }
    const int64_t parts = (int64_t)gridDim.x * blockDim.y, part = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int which[3] = {a.sum_gain, a.sum_post, a.sum_gate};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        if (which[k] < 0) continue;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int i = threadIdx.x + v * blockDim.x;
            if (i < vecs)
                store8<BQ_DT_F32>(reinterpret_cast<uint8_t*>(a.part + (which[k] * parts + part) * a.H), i, 0, sums[k][v]);
        }
    }
}

struct SumArgs {
    const float* part;   // [arrays][parts][H]
    int64_t parts;
    int H;
    float* out[3];
};

constexpr int kSumThreads = 512;

// The parts of 32 columns of one array (blockIdx.y) added up, each warp a share of them.
__global__ void __launch_bounds__(kSumThreads)
sum_parts_kernel(const SumArgs a) {
    constexpr int kWarps = kSumThreads / 32;
    __shared__ float s_red[kWarps][32];
    bq::grid_dependency_wait();
    bq::allow_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    const float* part = a.part + (int64_t)blockIdx.y * a.parts * a.H;
    float sum = 0.f;
    if (c < a.H) {
#pragma unroll 8
        for (int64_t i = warp; i < a.parts; i += kWarps) sum += part[i * a.H + c];
    }
    s_red[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && c < a.H) {
#pragma unroll
        for (int w = 1; w < kWarps; ++w) sum += s_red[w][lane];
        a.out[blockIdx.y][c] = sum;
    }
}

// ---------------------------------------------------------------- host side
bq_status check_desc(const char* name, const bq_residual_norm_desc* d, bool x) {
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
    if (d->gate_kind == BQ_GATE_FULL) return bq::check_rows(name, "gate", d->gate, d->H, d->ldgate, es);
    if (!bq::aligned(d->gate, d->gate_kind == BQ_GATE_CHANNEL ? 16 : es))
        return bq::fail(BQ_ERR_ALIGN, "%s: the gate is not aligned", name);
    return BQ_OK;
}

Rows rows(const void* p, int64_t ld, int32_t dtype) {
    return {static_cast<uint8_t*>(const_cast<void*>(p)), ld * bq::dtype_size(dtype), dtype};
}

Gate gate_of(const bq_residual_norm_desc* d) {
    return {static_cast<const uint8_t*>(d->gate), d->ldgate * bq::dtype_size(d->gate_dtype), d->gate_dtype, d->gate_kind,
            d->gate_sigmoid};
}

// Calls f with the row types as constants where all three are the same, else with kAny.
template <typename F>
void with_types(int dy, int dh, int dx, F f) {
    if (dy == dh && dh == dx) {
        if (dy == BQ_DT_F32) f(std::integral_constant<int, BQ_DT_F32>());
        else if (dy == BQ_DT_F16) f(std::integral_constant<int, BQ_DT_F16>());
        else f(std::integral_constant<int, BQ_DT_BF16>());
    } else {
        f(std::integral_constant<int, kAny>());
    }
}

// Threads of a row: at most `most`, the vectors shared evenly among as many as it takes.
struct RowShape {
    int threads, per_thread;   // per_thread a power of two
};

RowShape row_shape(int vecs, int most) {
    int per = 1;
    while ((vecs + per - 1) / per > most) per *= 2;
    return {((vecs + per - 1) / per + 31) / 32 * 32, per};
}

bq_status launched(const char* name, cudaError_t e) {
    if (e != cudaSuccess) {
        cudaGetLastError();   // reported here
        return bq::fail(BQ_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
    }
    bq::note_launch();
    return bq::check_launch(name);
}

// CTAs of the backward pass, and their row groups' column sums.
struct BackwardShape {
    RowShape row;
    int rows, ctas;
    size_t parts() const { return (size_t)rows * ctas; }
};

BackwardShape backward_shape(int T, int H) {
    BackwardShape b;
    b.row = row_shape(H / 8, kBackwardThreads);
    b.rows = std::max(1, kBackwardThreads / b.row.threads);
    b.ctas = (int)std::min<int64_t>(2 * kSms, ((int64_t)T + b.rows - 1) / b.rows);
    return b;
}

}  // namespace

extern "C" bq_status bq_residual_norm(const bq_residual_norm_desc* d, const void* y, int64_t ldy, const void* h,
                                      int64_t ldh, void* h_out, int64_t ldho, void* x, int64_t ldx,
                                      bq_stream_t stream) {
    const char* name = "bq_residual_norm";
    bq_status s = check_desc(name, d, x != nullptr);
    if (s != BQ_OK || d->T == 0) return s;
    const int ys = bq::dtype_size(d->y_dtype), hs = bq::dtype_size(d->h_dtype);
    if ((s = bq::check_rows(name, "y", y, d->H, ldy, ys)) != BQ_OK ||
        (s = bq::check_rows(name, "h", h, d->H, ldh, hs)) != BQ_OK ||
        (s = bq::check_rows(name, "h_out", h_out, d->H, ldho, hs)) != BQ_OK)
        return s;
    if (x && (s = bq::check_rows(name, "x", x, d->H, ldx, bq::dtype_size(d->x_dtype))) != BQ_OK) return s;
    if ((s = bq::check_arch()) != BQ_OK) return s;
    const int32_t x_dtype = x ? d->x_dtype : d->h_dtype;
    const ForwardArgs a{d->T, d->H, rows(y, ldy, d->y_dtype), rows(h, ldh, d->h_dtype), rows(h_out, ldho, d->h_dtype),
                        rows(x, ldx, x_dtype), static_cast<const uint8_t*>(d->gain),
                        static_cast<const uint8_t*>(d->post_gain), d->gain_dtype, gate_of(d), d->scale,
                        d->residual_scale, d->eps};
    const RowShape r = row_shape(d->H / 8, kForwardThreads);
    const int per_cta = std::max(1, 256 / r.threads);
    const dim3 grid((unsigned)(((int64_t)d->T + per_cta - 1) / per_cta)), block(r.threads, per_cta);
    cudaError_t e = cudaSuccess;
    with_types(d->y_dtype, d->h_dtype, x_dtype, [&](auto type) {
        constexpr int D = decltype(type)::value;
        auto go = [&](auto kernel) { e = bq::launch_after(kernel, grid, block, 0, (cudaStream_t)stream, a); };
        if (r.per_thread == 1) go(residual_norm_kernel<D, D, D, 1>);
        else if (r.per_thread == 2) go(residual_norm_kernel<D, D, D, 2>);
        else go(residual_norm_kernel<D, D, D, 4>);
    });
    return launched(name, e);
}

extern "C" size_t bq_residual_norm_backward_workspace_bytes(int32_t T, int32_t H) {
    if (T < 0 || H < 8 || H % 8 || H > kMaxH) return 0;
    return std::max<size_t>(1, backward_shape(T, H).parts()) * H * 4 * 3;
}

extern "C" bq_status bq_residual_norm_backward(const bq_residual_norm_desc* d, const void* y, int64_t ldy,
                                               const void* h_out, int64_t ldho, const void* dh_out, int64_t lddho,
                                               const void* dx, int64_t lddx, void* dy, int64_t lddy, void* dh,
                                               int64_t lddh, float* dgain, float* dpost_gain, void* dgate,
                                               int64_t lddgate, void* workspace, size_t workspace_bytes,
                                               bq_stream_t stream) {
    const char* name = "bq_residual_norm_backward";
    bq_status s = check_desc(name, d, dx != nullptr);
    if (s != BQ_OK) return s;
    const bool channel = d->gate_kind == BQ_GATE_CHANNEL;
    if ((dgain && d->T > 0 && !dx) || (dpost_gain && d->T > 0 && !d->post_gain) || (dgate && d->gate_kind == BQ_GATE_NONE))
        return bq::fail(BQ_ERR_NULL, "%s: a gradient is asked for without what it belongs to (dgain: dx, dpost_gain: "
                                     "post_gain, dgate: gate)", name);
    if (!bq::aligned(dgain, 4) || !bq::aligned(dpost_gain, 4) ||
        (d->gate_kind != BQ_GATE_FULL && !bq::aligned(dgate, 4)))
        return bq::fail(BQ_ERR_ALIGN, "%s: sums must be 4-byte aligned", name);
    const bool sums = dgain || dpost_gain || (dgate && channel);
    if (d->T == 0 && !sums) return BQ_OK;
    if (d->T > 0) {
        const int ys = bq::dtype_size(d->y_dtype), hs = bq::dtype_size(d->h_dtype);
        if (!dx && !dh_out) return bq::fail(BQ_ERR_NULL, "%s: dx and dh_out are both NULL", name);
        if ((s = bq::check_rows(name, "y", y, d->H, ldy, ys)) != BQ_OK ||
            (dx && (s = bq::check_rows(name, "h_out", h_out, d->H, ldho, hs)) != BQ_OK) ||
            (dh_out && (s = bq::check_rows(name, "dh_out", dh_out, d->H, lddho, hs)) != BQ_OK) ||
            (dx && (s = bq::check_rows(name, "dx", dx, d->H, lddx, bq::dtype_size(d->x_dtype))) != BQ_OK) ||
            (s = bq::check_rows(name, "dy", dy, d->H, lddy, ys)) != BQ_OK ||
            (s = bq::check_rows(name, "dh", dh, d->H, lddh, hs)) != BQ_OK)
            return s;
        if (dgate && d->gate_kind == BQ_GATE_FULL &&
            (s = bq::check_rows(name, "dgate", dgate, d->H, lddgate, bq::dtype_size(d->gate_dtype))) != BQ_OK)
            return s;
    }
    const BackwardShape b = backward_shape(d->T, d->H);
    if (sums) {
        const size_t need = bq_residual_norm_backward_workspace_bytes(d->T, d->H);
        if (!workspace || workspace_bytes < need)
            return bq::fail(BQ_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu", name, workspace_bytes, need);
        if (!bq::aligned(workspace, 16)) return bq::fail(BQ_ERR_ALIGN, "%s: workspace must be 16-byte aligned", name);
    }
    if ((s = bq::check_arch()) != BQ_OK) return s;
    SumArgs sum{static_cast<const float*>(workspace), (int64_t)b.parts(), d->H, {nullptr, nullptr, nullptr}};
    int arrays = 0;
    auto array_of = [&](void* out) {
        if (!out) return -1;
        sum.out[arrays] = static_cast<float*>(out);
        return arrays++;
    };
    const int i_gain = array_of(dgain), i_post = array_of(dpost_gain), i_gate = array_of(channel ? dgate : nullptr);
    cudaStream_t st = (cudaStream_t)stream;
    if (d->T > 0) {
        const int32_t x_dtype = dx ? d->x_dtype : d->h_dtype;
        const BackwardArgs a{d->T, d->H, rows(y, ldy, d->y_dtype), rows(h_out, ldho, d->h_dtype),
                             rows(dh_out, lddho, d->h_dtype), rows(dx, lddx, x_dtype), rows(dy, lddy, d->y_dtype),
                             rows(dh, lddh, d->h_dtype), static_cast<const uint8_t*>(d->gain),
                             static_cast<const uint8_t*>(d->post_gain), d->gain_dtype, gate_of(d),
                             rows(dgate, lddgate, d->gate_dtype), d->scale, d->residual_scale, d->eps,
                             static_cast<float*>(workspace), i_gain, i_post, i_gate};
        const dim3 grid(b.ctas), block(b.row.threads, b.rows);
        cudaError_t e = cudaSuccess;
        with_types(d->y_dtype, d->h_dtype, x_dtype, [&](auto type) {
            constexpr int D = decltype(type)::value;
            auto go = [&](auto kernel) { e = bq::launch_after(kernel, grid, block, 0, st, a); };
            if (b.row.per_thread == 1) go(residual_norm_backward_kernel<D, D, D, 1>);
            else if (b.row.per_thread == 2) go(residual_norm_backward_kernel<D, D, D, 2>);
            else if (b.row.per_thread == 4) go(residual_norm_backward_kernel<D, D, D, 4>);
            else go(residual_norm_backward_kernel<D, D, D, 8>);
        });
        if ((s = launched(name, e)) != BQ_OK) return s;
    }
    if (!sums) return BQ_OK;
    return launched(name, bq::launch_after(sum_parts_kernel, dim3((d->H + 31) / 32, arrays), dim3(kSumThreads), 0, st, sum));
}
