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
#include <atomic>

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
    int dtype, kind, sigmoid;
};

// Two fp32 values in a register pair: the packed instructions do both in one issue slot, and these kernels would be
// bound by issue without them.
typedef unsigned long long f32x2;

__device__ __forceinline__ f32x2 two(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ f32x2 both(float v) { return two(v, v); }

__device__ __forceinline__ float2 parts_of(f32x2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}

__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ float sum2(f32x2 v) {
    const float2 p = parts_of(v);
    return p.x + p.y;
}

// Eight values of a row.
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
__device__ __forceinline__ Vec load8(const uint8_t* row, int i, int dtype) {
    const uint4* p = reinterpret_cast<const uint4*>(row) + (dtype == BQ_DT_F32 ? 2 * i : i);
    return unpack8<kAny>(p[0], dtype == BQ_DT_F32 ? p[1] : p[0], dtype);
}

template <int DT>
__device__ __forceinline__ void store8(uint8_t* to, int dtype, const Vec& v) {
    const int dt = DT == kAny ? dtype : DT;
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 x = parts_of(v.p[j]);
        f[2 * j] = x.x;
        f[2 * j + 1] = x.y;
    }
    if (dt == BQ_DT_F32) {
        reinterpret_cast<float4*>(to)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(to)[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        *reinterpret_cast<uint4*>(to) = dt == BQ_DT_F16 ? bq::RowVec<BQ_DT_F16>::pack(f) : bq::RowVec<BQ_DT_BF16>::pack(f);
    }
}

__device__ __forceinline__ float load1(const uint8_t* p, int64_t i, int dtype) {
    if (dtype == BQ_DT_F32) return reinterpret_cast<const float*>(p)[i];
    if (dtype == BQ_DT_F16) return __half2float(reinterpret_cast<const __half*>(p)[i]);
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}

__device__ __forceinline__ float sigmoid_f(float v) { return 1.f / (1.f + expf(-v)); }

__device__ __forceinline__ Vec sigmoid8(const Vec& v) {
    Vec r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 x = parts_of(v.p[j]);
        r.p[j] = two(sigmoid_f(x.x), sigmoid_f(x.y));
    }
    return r;
}

// ---------------------------------------------------------------- rows in flight
// Each thread fetches the vectors that it will use itself, rows ahead, into shared memory of its own (cp.async, 16
// bytes at a time): the loads need no registers while they are in flight, and no barrier when they land.
constexpr int kMaxThreads = 512;
constexpr int kMaxArrays = 5;

struct Staged {
    const uint8_t* p;    // NULL: not there
    int64_t ld, advance; // bytes of a row, and of the rows that a block steps over
    int dtype;
    int at;              // where its rows lie in a stage: a plane of 16 bytes per vector, or two (fp32), so that a
                         // warp's vectors lie in distinct banks
};

struct Ring {
    Staged array[kMaxArrays];
    int stages, stage_bytes;
    int plane;         // bytes of a plane: 16 of every vector of the block's rows
    int vecs, slice;   // vectors of a row, and of a row in this CTA (a cluster shares a row)
};

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

__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Which vectors of a row a thread has: x, x + blockDim.x, ... of the CTA's.
template <int VPT>
struct Mine {
    int v0;              // first vector of the CTA's slice
    int at;              // bytes of the thread's first vector into a plane
    bool has[VPT];

    __device__ __forceinline__ Mine(const Ring& g, int rank) {
        v0 = rank * g.slice;
        at = (threadIdx.y * g.slice + threadIdx.x) * 16;
        const int n = min(g.slice, g.vecs - v0);
#pragma unroll
        for (int v = 0; v < VPT; ++v) has[v] = (int)(threadIdx.x + v * blockDim.x) < n;
    }
    __device__ __forceinline__ int vec(int v) const { return v0 + threadIdx.x + v * blockDim.x; }
    __device__ __forceinline__ int place(int v) const { return at + v * (int)blockDim.x * 16; }   // in a plane
};

__device__ __forceinline__ int vec_bytes(int dtype) { return dtype == BQ_DT_F32 ? 32 : 16; }

// Where a thread's vectors of a matrix lie, row after row of its block.
struct Walk {
    uint8_t* p;

    template <int VPT>
    __device__ __forceinline__ Walk(const uint8_t* base, int64_t ld, int dtype, int64_t row, const Mine<VPT>& m)
        : p(const_cast<uint8_t*>(base) + row * ld + (int64_t)m.vec(0) * vec_bytes(dtype)) {}
};

template <int DT, int VPT>
__device__ __forceinline__ void fetch(const Ring& g, int k, Walk& from, uint32_t stage, bool live, const Mine<VPT>& m) {
    const Staged& a = g.array[k];
    if (!a.p) return;
    const bool wide = (DT == kAny ? a.dtype : DT) == BQ_DT_F32;
    if (live) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            if (!m.has[v]) continue;
            const uint32_t dst = stage + a.at + m.place(v);
            const uint8_t* src = from.p + v * (int)blockDim.x * (wide ? 32 : 16);
            copy16_async(dst, src);
            if (wide) copy16_async(dst + g.plane, src + 16);
        }
    }
    from.p += a.advance;
}

__device__ __forceinline__ void end_of_row() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Waits for the oldest row in flight (stages - 1 of them are).
__device__ __forceinline__ void row_landed(int stages) {
    if (stages == 2) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else asm volatile("cp.async.wait_group 1;" ::: "memory");
}

// A vector of array k in a stage.
template <int DT>
__device__ __forceinline__ Vec staged8(const Ring& g, const uint8_t* stage, int k, int place) {
    const uint8_t* p = stage + g.array[k].at + place;
    const int dtype = g.array[k].dtype;
    const uint4 lo = *reinterpret_cast<const uint4*>(p);
    if ((DT == kAny ? dtype : DT) != BQ_DT_F32) return unpack8<DT>(lo, lo, dtype);
    return unpack8<BQ_DT_F32>(lo, *reinterpret_cast<const uint4*>(p + g.plane), dtype);
}

enum { kGain = 0, kBranch = 1 };   // a thread's column constants, fp32: gain; scale * post_gain * (a gate per channel)

__device__ __forceinline__ void keep8(const Ring& g, uint8_t* s_const, int which, int place, const Vec& v) {
    uint8_t* p = s_const + 2 * which * g.plane + place;
    *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(v.p[0], v.p[1]);
    *reinterpret_cast<ulonglong2*>(p + g.plane) = make_ulonglong2(v.p[2], v.p[3]);
}

__device__ __forceinline__ Vec kept8(const Ring& g, const uint8_t* s_const, int which, int place) {
    const uint8_t* p = s_const + 2 * which * g.plane + place;
    const ulonglong2 lo = *reinterpret_cast<const ulonglong2*>(p), hi = *reinterpret_cast<const ulonglong2*>(p + g.plane);
    return {{lo.x, lo.y, hi.x, hi.y}};
}

struct Columns {
    const uint8_t *gain, *post;        // NULL: none
    int gain_dtype;
    Gate gate;
    float scale;
};

// The constants of a thread's own columns, while its first rows are on their way.
template <int VPT>
__device__ __forceinline__ void keep_columns(const Ring& g, uint8_t* s_const, const Columns& c, const Mine<VPT>& m) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        if (!m.has[v]) continue;
        if (c.gain) keep8(g, s_const, kGain, m.place(v), load8(c.gain, m.vec(v), c.gain_dtype));
        Vec b = same8(c.scale);
        if (c.post) {
            const Vec p = load8(c.post, m.vec(v), c.gain_dtype);
#pragma unroll
            for (int j = 0; j < 4; ++j) b.p[j] = mul2(b.p[j], p.p[j]);
        }
        if (c.gate.kind == GATE_CHANNEL) {
            Vec f = load8(c.gate.p, m.vec(v), c.gate.dtype);
            if (c.gate.sigmoid) f = sigmoid8(f);
#pragma unroll
            for (int j = 0; j < 4; ++j) b.p[j] = mul2(b.p[j], f.p[j]);
        }
        keep8(g, s_const, kBranch, m.place(v), b);
    }
}

// The factor that a row's branch has as a whole: a gate per token, or 1.
__device__ __forceinline__ float token_factor(const Gate& gate, int64_t t, bool live) {
    if (!live || gate.kind != GATE_TOKEN) return 1.f;
    const float f = load1(gate.p, t, gate.dtype);
    return gate.sigmoid ? sigmoid_f(f) : f;
}

// What the sums over a row go through.  Consecutive sums take different halves, so a half is written again only
// behind the barrier of the sum between.
struct SumBuf {
    float warp[2][kMaxThreads / 32][4];
    float cta[2][4];
};

// N sums over the threads of a row, the same in each: lanes and warps by butterflies, CTAs in order.
template <int N, bool CLUSTER>
__device__ __forceinline__ void row_sums(float (&v)[N], SumBuf& buf, int& turn, int ranks) {
    static_assert(N <= 4, "");
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int off = 16; off; off >>= 1) v[n] += __shfl_xor_sync(0xffffffffu, v[n], off);
    const int warps = blockDim.x >> 5;
    if (warps == 1 && !CLUSTER) return;
    float (*mine)[4] = buf.warp[turn] + threadIdx.y * warps;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int n = 0; n < N; ++n) mine[threadIdx.x >> 5][n] = v[n];
    }
    __syncthreads();
    if (!CLUSTER || threadIdx.x < 32) {
        // the warps' sums (16 at most), one a lane, by a butterfly again
        const int w = threadIdx.x & 15;
        const float4 f = w < warps ? *reinterpret_cast<const float4*>(mine[w]) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float x[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int n = 0; n < N; ++n) {
            v[n] = x[n];
#pragma unroll
            for (int off = 8; off; off >>= 1) v[n] += __shfl_xor_sync(0xffffffffu, v[n], off);
        }
    }
    if (CLUSTER) {
        if (threadIdx.x == 0) {
#pragma unroll
            for (int n = 0; n < N; ++n) buf.cta[turn][n] = v[n];
        }
        cluster_sync();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            v[n] = 0.f;
            for (int r = 0; r < ranks; ++r) v[n] += peer_load(&buf.cta[turn][n], r);
        }
    }
    turn ^= 1;
}

// ---------------------------------------------------------------- forward
struct ForwardArgs {
    int T, H;
    Ring ring;                      // y, h and a gate per value
    Rows out, x;                    // x.p NULL: not computed
    int64_t out_advance, x_advance;
    Columns columns;
    float residual_scale, eps;
};

// blockDim.x threads take a row (or a cluster's slice of one), a thread the vectors x, x + blockDim.x, ... of it;
// blockDim.y rows at a time.
template <int DY, int DH, int DX, int VPT, bool CLUSTER>
__global__ void __launch_bounds__(kMaxThreads)
residual_norm_kernel(const __grid_constant__ ForwardArgs a) {
    extern __shared__ __align__(16) uint8_t s_ring[];
    __shared__ SumBuf s_buf;
    bq::grid_dependency_wait();   // launched behind whatever precedes it on the stream
    bq::allow_dependents();
    const Ring& g = a.ring;
    const Gate& gate = a.columns.gate;
    const bool post = a.columns.post != nullptr;
    const int ranks = CLUSTER ? (g.vecs + g.slice - 1) / g.slice : 1, rank = CLUSTER ? (int)cluster_rank() : 0;
    const Mine<VPT> m(g, rank);
    const int64_t block0 = (int64_t)(blockIdx.x / ranks) * blockDim.y, step = (int64_t)(gridDim.x / ranks) * blockDim.y;
    const int64_t first = block0 + threadIdx.y;
    Walk y(g.array[0].p, g.array[0].ld, g.array[0].dtype, first, m), h(g.array[1].p, g.array[1].ld, g.array[1].dtype, first, m);
    Walk w(g.array[2].p, g.array[2].ld, g.array[2].dtype, first, m);
    Walk out(a.out.p, a.out.ld, a.out.dtype, first, m), x(a.x.p, a.x.ld, a.x.dtype, first, m);
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(s_ring);
    uint8_t* s_const = s_ring + g.stages * g.stage_bytes;
    auto fetch_row = [&](int stage, int64_t t) {
        const uint32_t to = ring + stage * g.stage_bytes;
        const bool live = t < a.T;
        fetch<DY>(g, 0, y, to, live, m);
        fetch<DH>(g, 1, h, to, live, m);
        fetch<kAny>(g, 2, w, to, live, m);
        end_of_row();
    };
    for (int i = 0; i < g.stages - 1; ++i) fetch_row(i, first + i * step);
    keep_columns(g, s_const, a.columns, m);
    int stage = 0, ahead = g.stages - 1, turn = 0;
    const float inv_h = 1.f / (float)a.H;
    for (int64_t t0 = block0; t0 < a.T; t0 += step) {
        const int64_t t = t0 + threadIdx.y;
        const bool live = t < a.T;
        row_landed(g.stages);
        fetch_row(ahead, t + (g.stages - 1) * step);
        const uint8_t* s = s_ring + stage * g.stage_bytes;
        if (++ahead == g.stages) ahead = 0;
        if (++stage == g.stages) stage = 0;
        float f = token_factor(gate, t, live);
        Vec r[VPT];
        if (post) {
            f32x2 squares = both(0.f);
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                if (!live || !m.has[v]) continue;
                r[v] = staged8<DY>(g, s, 0, m.place(v));
#pragma unroll
                for (int j = 0; j < 4; ++j) squares = fma2(r[v].p[j], r[v].p[j], squares);
            }
            float sum[1] = {sum2(squares)};
            row_sums<1, CLUSTER>(sum, s_buf, turn, ranks);
            f *= rsqrtf(__fmaf_rn(sum[0], inv_h, a.eps));
        }
        f32x2 squares = both(0.f);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            if (!live || !m.has[v]) continue;
            if (!post) r[v] = staged8<DY>(g, s, 0, m.place(v));
            const Vec c = kept8(g, s_const, kBranch, m.place(v)), o = staged8<DH>(g, s, 1, m.place(v));
            if (gate.kind == GATE_FULL) {
                Vec k = staged8<kAny>(g, s, 2, m.place(v));
                if (gate.sigmoid) k = sigmoid8(k);
#pragma unroll
                for (int j = 0; j < 4; ++j) r[v].p[j] = mul2(r[v].p[j], k.p[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                r[v].p[j] = fma2(mul2(r[v].p[j], both(f)), c.p[j], mul2(o.p[j], both(a.residual_scale)));
                squares = fma2(r[v].p[j], r[v].p[j], squares);
            }
            store8<DH>(out.p + v * (int)blockDim.x * vec_bytes(DH == kAny ? a.out.dtype : DH), a.out.dtype, r[v]);
        }
        out.p += a.out_advance;
        if (!a.x.p) continue;
        float sum[1] = {sum2(squares)};
        row_sums<1, CLUSTER>(sum, s_buf, turn, ranks);
        const float norm = rsqrtf(__fmaf_rn(sum[0], inv_h, a.eps));
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            if (!live || !m.has[v]) continue;
            const Vec c = kept8(g, s_const, kGain, m.place(v));
#pragma unroll
            for (int j = 0; j < 4; ++j) r[v].p[j] = mul2(mul2(r[v].p[j], both(norm)), c.p[j]);
            store8<DX>(x.p + v * (int)blockDim.x * vec_bytes(DX == kAny ? a.x.dtype : DX), a.x.dtype, r[v]);
        }
        x.p += a.x_advance;
    }
    if (CLUSTER) cluster_sync();   // peers may still be reading this CTA's sums
}

// ---------------------------------------------------------------- backward
// With P = scale * post_gain * (a gate per channel), f the gate per token and w the one per value (or 1 each),
// yn = s y (y without a post norm), all of it per column or row, the formulas at the top become
//   dy = f (s P w G - y s^3 mean(P w G y)), or f P w G;   Q = sum over rows of f w G yn
//   dpost_gain = scale gate Q;   dgate per channel = scale gate' post_gain Q
//   dgate per token = gate' mean-sum of P G yn;   dgate per value = P G yn w'
// so one column sum serves both gradients of the branch, and the constants are folded in at the end.
enum { kY = 0, kOut = 1, kDx = 2, kDout = 3, kFull = 4 };

struct BackwardArgs {
    int T, H;
    Ring ring;                      // y, h', dx, dh' and a gate per value, those there are (kOut ...)
    Rows dy, dh;
    Columns columns;
    Rows dgate;                     // of a gate per token (fp32) or per value; p NULL: not computed
    int64_t dy_advance, dh_advance, dgate_advance;
    float residual_scale, eps;
    float* part;                    // [arrays][parts][H] column sums: dgain, Q
    int sum_gain, sum_branch;       // which array each is, or -1
};

// Blocks walk over the rows; a thread's columns stay the same, so it adds their column sums in registers.
template <int DY, int DH, int DX, int VPT, bool CLUSTER>
__global__ void __launch_bounds__(kMaxThreads)
residual_norm_backward_kernel(const __grid_constant__ BackwardArgs a) {
    extern __shared__ __align__(16) uint8_t s_ring[];
    __shared__ SumBuf s_buf;
    bq::grid_dependency_wait();   // launched behind whatever precedes it on the stream
    bq::allow_dependents();
    const Ring& g = a.ring;
    const Gate& gate = a.columns.gate;
    const bool post = a.columns.post != nullptr, has_x = g.array[kDx].p != nullptr, branch_sum = a.sum_branch >= 0;
    const int ranks = CLUSTER ? (g.vecs + g.slice - 1) / g.slice : 1, rank = CLUSTER ? (int)cluster_rank() : 0;
    const Mine<VPT> m(g, rank);
    const int64_t block0 = (int64_t)(blockIdx.x / ranks) * blockDim.y, step = (int64_t)(gridDim.x / ranks) * blockDim.y;
    const int64_t first = block0 + threadIdx.y;
    auto walk = [&](int k) { return Walk(g.array[k].p, g.array[k].ld, g.array[k].dtype, first, m); };
    Walk w_y = walk(kY), w_out = walk(kOut), w_dx = walk(kDx), w_dout = walk(kDout), w_gate = walk(kFull);
    Walk dy(a.dy.p, a.dy.ld, a.dy.dtype, first, m), dh(a.dh.p, a.dh.ld, a.dh.dtype, first, m);
    Walk dgate(a.dgate.p, a.dgate.ld, a.dgate.dtype, first, m);
    const int dy_next = blockDim.x * vec_bytes(DY == kAny ? a.dy.dtype : DY);
    const int dh_next = blockDim.x * vec_bytes(DH == kAny ? a.dh.dtype : DH);
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(s_ring);
    uint8_t* s_const = s_ring + g.stages * g.stage_bytes;
    auto fetch_row = [&](int stage, int64_t t) {
        const uint32_t to = ring + stage * g.stage_bytes;
        const bool live = t < a.T;
        fetch<DY>(g, kY, w_y, to, live, m);
        fetch<DH>(g, kOut, w_out, to, live, m);
        fetch<DX>(g, kDx, w_dx, to, live, m);
        fetch<DH>(g, kDout, w_dout, to, live, m);
        fetch<kAny>(g, kFull, w_gate, to, live, m);
        end_of_row();
    };
    for (int i = 0; i < g.stages - 1; ++i) fetch_row(i, first + i * step);
    keep_columns(g, s_const, a.columns, m);
    int stage = 0, ahead = g.stages - 1, turn = 0;
    Vec gain_sum[VPT], branch[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) gain_sum[v] = branch[v] = same8(0.f);
    const float inv_h = 1.f / (float)a.H;
    for (int64_t t0 = block0; t0 < a.T; t0 += step) {
        const int64_t t = t0 + threadIdx.y;
        const bool live = t < a.T;
        row_landed(g.stages);
        fetch_row(ahead, t + (g.stages - 1) * step);
        const uint8_t* st = s_ring + stage * g.stage_bytes;
        if (++ahead == g.stages) ahead = 0;
        if (++stage == g.stages) stage = 0;
        const float f = token_factor(gate, t, live);
        float r = 0.f, c = 0.f, s = 1.f;
        Vec h[VPT], d[VPT], y[VPT];
        if (has_x || post) {
            f32x2 hh = both(0.f), dh = both(0.f), yy = both(0.f);
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                if (!live || !m.has[v]) continue;
                if (has_x) {
                    h[v] = staged8<DH>(g, st, kOut, m.place(v));
                    d[v] = staged8<DX>(g, st, kDx, m.place(v));
                    const Vec k = kept8(g, s_const, kGain, m.place(v));
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        hh = fma2(h[v].p[j], h[v].p[j], hh);
                        dh = fma2(mul2(d[v].p[j], k.p[j]), h[v].p[j], dh);
                    }
                }
                if (post) {
                    y[v] = staged8<DY>(g, st, kY, m.place(v));
#pragma unroll
                    for (int j = 0; j < 4; ++j) yy = fma2(y[v].p[j], y[v].p[j], yy);
                }
            }
            float sums[3] = {sum2(hh), sum2(dh), sum2(yy)};
            row_sums<3, CLUSTER>(sums, s_buf, turn, ranks);
            r = rsqrtf(__fmaf_rn(sums[0], inv_h, a.eps));
            c = -r * r * r * (sums[1] * inv_h);
            if (post) s = rsqrtf(__fmaf_rn(sums[2], inv_h, a.eps));
        }
        const float fs = f * s;
        f32x2 inner = both(0.f);         // P w G y
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            if (!live || !m.has[v]) continue;
            Vec G = g.array[kDout].p ? staged8<DH>(g, st, kDout, m.place(v)) : same8(0.f);
            if (has_x) {
                const Vec k = kept8(g, s_const, kGain, m.place(v));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x2 dr = mul2(d[v].p[j], both(r));
                    gain_sum[v].p[j] = fma2(dr, h[v].p[j], gain_sum[v].p[j]);
                    G.p[j] = fma2(h[v].p[j], both(c), fma2(k.p[j], dr, G.p[j]));
                }
            }
            Vec o;
#pragma unroll
            for (int j = 0; j < 4; ++j) o.p[j] = mul2(G.p[j], both(a.residual_scale));
            store8<DH>(dh.p + v * dh_next, a.dh.dtype, o);
            const Vec p = kept8(g, s_const, kBranch, m.place(v));
            if (!post) y[v] = staged8<DY>(g, st, kY, m.place(v));
            if (gate.kind == GATE_FULL) {
                Vec w = staged8<kAny>(g, st, kFull, m.place(v)), dw;
#pragma unroll
                for (int j = 0; j < 4; ++j) dw.p[j] = mul2(mul2(G.p[j], p.p[j]), mul2(y[v].p[j], both(s)));
                if (gate.sigmoid) {
                    w = sigmoid8(w);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        dw.p[j] = mul2(dw.p[j], mul2(w.p[j], fma2(w.p[j], both(-1.f), both(1.f))));
                }
                if (a.dgate.p)
                    store8<kAny>(dgate.p + v * (int)blockDim.x * vec_bytes(a.dgate.dtype), a.dgate.dtype, dw);
#pragma unroll
                for (int j = 0; j < 4; ++j) G.p[j] = mul2(G.p[j], w.p[j]);
            }
            if (branch_sum) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    branch[v].p[j] = fma2(mul2(G.p[j], both(fs)), y[v].p[j], branch[v].p[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                G.p[j] = mul2(G.p[j], p.p[j]);
                inner = fma2(G.p[j], y[v].p[j], inner);
            }
            if (post) {
                d[v] = G;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) G.p[j] = mul2(G.p[j], both(f));
                store8<DY>(dy.p + v * dy_next, a.dy.dtype, G);
            }
        }
        uint8_t* to_dy = dy.p;
        dh.p += a.dh_advance;
        dy.p += a.dy_advance;
        dgate.p += a.dgate_advance;
        if (!post && !(gate.kind == GATE_TOKEN && a.dgate.p)) continue;
        float sums[1] = {sum2(inner)};
        row_sums<1, CLUSTER>(sums, s_buf, turn, ranks);
        if (gate.kind == GATE_TOKEN && a.dgate.p && live && threadIdx.x == 0 && rank == 0)
            reinterpret_cast<float*>(a.dgate.p)[t] = s * sums[0] * (gate.sigmoid ? f * (1.f - f) : 1.f);
        if (!post) continue;
        const float cy = -f * s * s * s * (sums[0] * inv_h);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            if (!live || !m.has[v]) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) d[v].p[j] = fma2(y[v].p[j], both(cy), mul2(d[v].p[j], both(fs)));
            store8<DY>(to_dy + v * dy_next, a.dy.dtype, d[v]);
        }
    }
    // the block's column sums: its rows added up in shared memory (the ring is free), then to its part
    const int64_t parts = gridDim.x / ranks, part = blockIdx.x / ranks;
    const int which[2] = {a.sum_gain, a.sum_branch};
    float* s_sum = reinterpret_cast<float*>(s_ring);
    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (which[k] < 0) continue;
        uint8_t* out = reinterpret_cast<uint8_t*>(a.part + (which[k] * parts + part) * a.H);
        if (blockDim.y > 1) __syncthreads();
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            if (!m.has[v]) continue;
            const Vec& sum = k ? branch[v] : gain_sum[v];
            if (blockDim.y == 1) store8<BQ_DT_F32>(out + (int64_t)m.vec(v) * 32, 0, sum);
            else store8<BQ_DT_F32>(s_ring + 2 * m.place(v), 0, sum);
        }
        if (blockDim.y == 1) continue;
        __syncthreads();
        for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < g.vecs * 8; i += blockDim.x * blockDim.y) {
            float sum = 0.f;   // blocks of several rows are not clusters: the slice is the row
            for (int y = 0; y < (int)blockDim.y; ++y) sum += s_sum[y * g.slice * 8 + i];
            reinterpret_cast<float*>(out)[i] = sum;
        }
    }
    if (CLUSTER) cluster_sync();   // peers may still be reading this CTA's sums
}

struct SumArgs {
    const float* part;   // [arrays][parts][H]
    int64_t parts;
    int H;
    float *dgain, *dpost, *dgate;     // NULL: not computed
    int sum_gain, sum_branch;
    Columns columns;
};

constexpr int kSumThreads = 512;

// The parts of 32 columns of one array (blockIdx.y) added up, each warp a share of them, and its gradients' constants.
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
    if (warp || c >= a.H) return;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) sum += s_red[w][lane];
    if ((int)blockIdx.y == a.sum_gain) {
        a.dgain[c] = sum;
        return;
    }
    sum *= a.columns.scale;
    const Gate& gate = a.columns.gate;
    float f = 1.f, df = 1.f;
    if (gate.kind == GATE_CHANNEL) {
        f = load1(gate.p, c, gate.dtype);
        if (gate.sigmoid) {
            f = sigmoid_f(f);
            df = f * (1.f - f);
        }
    }
    if (a.dpost) a.dpost[c] = a.parts ? sum * f : 0.f;
    if (a.dgate) a.dgate[c] = a.parts ? sum * df * (a.columns.post ? load1(a.columns.post, c, a.columns.gain_dtype) : 1.f) : 0.f;
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

Columns columns_of(const bq_residual_norm_desc* d, bool x) {
    const Gate gate{static_cast<const uint8_t*>(d->gate), d->gate_dtype, d->gate_kind, d->gate_sigmoid};
    return {x ? static_cast<const uint8_t*>(d->gain) : nullptr, static_cast<const uint8_t*>(d->post_gain), d->gain_dtype,
            gate, d->scale};
}

template <int Y, int H, int X>
struct Types {
    static constexpr int y = Y, h = H, x = X;
};

// Calls f with the row types as constants: one type for all, a 16-bit type with an fp32 block output (as this
// library's MoE layer leaves it) or with an fp32 stream; other mixes read their types from the arguments.
template <typename F>
void with_types(int y, int h, int x, F f) {
    constexpr int F32 = BQ_DT_F32, F16 = BQ_DT_F16, BF16 = BQ_DT_BF16;
    if (y == F32 && h == F32 && x == F32) f(Types<F32, F32, F32>());
    else if (y == F16 && h == F16 && x == F16) f(Types<F16, F16, F16>());
    else if (y == BF16 && h == BF16 && x == BF16) f(Types<BF16, BF16, BF16>());
    else if (y == F32 && h == F16 && x == F16) f(Types<F32, F16, F16>());
    else if (y == F32 && h == BF16 && x == BF16) f(Types<F32, BF16, BF16>());
    else if (y == F16 && h == F32 && x == F16) f(Types<F16, F32, F16>());
    else if (y == BF16 && h == F32 && x == BF16) f(Types<BF16, F32, BF16>());
    else f(Types<kAny, kAny, kAny>());
}

// How a call's rows are spread: a cluster of CTAs per row, threads per row and vectors of each, rows of a block, rows
// in flight.
struct Shape {
    int cluster, slice, threads, per_thread, rows, stages, blocks;   // blocks: clusters in the grid
    size_t smem;
};

constexpr int kConstantBytes = 64;   // per vector: two constants of eight fp32

constexpr int kMaxBlocks = 2 * kSms;
constexpr size_t kSmemOfSm = 224 * 1024;

// bytes: of the staged arrays, per vector of eight values.
Shape shape_of(int T, int H, int bytes) {
    Shape p;
    const int vecs = H / 8;
    // a CTA holds up to 1024 vectors of a row, and two rows of it
    p.cluster = 1;
    while ((vecs + p.cluster - 1) / p.cluster > 2 * kMaxThreads ||
           (size_t)((vecs + p.cluster - 1) / p.cluster) * (2 * bytes + kConstantBytes) > kSmemOfSm)
        p.cluster *= 2;
    p.slice = (vecs + p.cluster - 1) / p.cluster;
    p.per_thread = p.slice > 256 ? 2 : 1;
    p.threads = ((p.slice + p.per_thread - 1) / p.per_thread + 31) / 32 * 32;
    p.rows = p.cluster > 1 ? 1 : std::max(1, 256 / p.threads);
    const size_t stage = (size_t)p.rows * p.slice * bytes, constants = (size_t)p.rows * p.slice * kConstantBytes;
    // two CTAs an SM where two rows of each fit, with a third row where that fits too
    const int per_sm = p.threads <= 256 && 2 * stage + constants <= kSmemOfSm / 2 ? 2 : 1;
    p.stages = 3 * stage + constants <= kSmemOfSm / per_sm ? 3 : 2;
    p.smem = p.stages * stage + constants;   // room for the block's column sums too, 32 bytes per vector
    // clusters of 1, 2, 4 and 8 CTAs that this GPU holds at once, with one CTA an SM
    const int held = p.cluster == 1 ? kSms : p.cluster == 2 ? 76 : p.cluster == 4 ? 36 : 15;
    p.blocks = (int)std::min<int64_t>(held * per_sm, ((int64_t)T + p.rows - 1) / p.rows);
    return p;
}

// The ring of a call: arrays are put in their places, then laid out.
struct RingMaker {
    Ring g{};
    int bytes = 0;
    void put(int k, const void* p, int64_t ld, int32_t dtype) {
        const int es = bq::dtype_size(dtype);
        g.array[k] = {static_cast<const uint8_t*>(p), ld * es, 0, dtype, 0};
        bytes += 8 * es;
    }
    Ring laid_out(const Shape& p, int H) {
        int at = 0;
        g.plane = p.rows * p.slice * 16;
        for (Staged& a : g.array) {
            if (!a.p) continue;
            a.at = at;
            a.advance = a.ld * p.rows * p.blocks;
            at += g.plane * (a.dtype == BQ_DT_F32 ? 2 : 1);
        }
        g.stages = p.stages;
        g.stage_bytes = at;
        g.vecs = H / 8;
        g.slice = p.slice;
        return g;
    }
};

template <auto kernel, typename Args>
cudaError_t launch_rows(const Shape& p, const Args& a, cudaStream_t st) {
    // per device: the attribute is a property of the function on the current device
    static std::atomic<bool> attr_set[64];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_set[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemOfSm);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.blocks * p.cluster));
    cfg.blockDim = dim3(p.threads, p.rows);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

bq_status launched(const char* name, cudaError_t e) {
    if (e != cudaSuccess) {
        cudaGetLastError();   // reported here
        return bq::fail(BQ_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
    }
    bq::note_launch();
    return bq::check_launch(name);
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
    RingMaker ring;
    ring.put(0, y, ldy, d->y_dtype);
    ring.put(1, h, ldh, d->h_dtype);
    if (d->gate_kind == BQ_GATE_FULL) ring.put(2, d->gate, d->ldgate, d->gate_dtype);
    const Shape p = shape_of(d->T, d->H, ring.bytes);
    const Rows out = rows(h_out, ldho, d->h_dtype), to_x = rows(x, ldx, x_dtype);
    const int64_t step = (int64_t)p.rows * p.blocks;
    const ForwardArgs a{d->T, d->H, ring.laid_out(p, d->H), out, to_x, out.ld * step, to_x.ld * step,
                        columns_of(d, x != nullptr), d->residual_scale, d->eps};
    cudaError_t e = cudaSuccess;
    with_types(d->y_dtype, d->h_dtype, x_dtype, [&](auto type) {
        using D = decltype(type);
        if (p.cluster > 1) e = p.per_thread == 1 ? launch_rows<residual_norm_kernel<kAny, kAny, kAny, 1, true>>(p, a, (cudaStream_t)stream)
                                              : launch_rows<residual_norm_kernel<kAny, kAny, kAny, 2, true>>(p, a, (cudaStream_t)stream);
        else if (p.per_thread == 1) e = launch_rows<residual_norm_kernel<D::y, D::h, D::x, 1, false>>(p, a, (cudaStream_t)stream);
        else e = launch_rows<residual_norm_kernel<D::y, D::h, D::x, 2, false>>(p, a, (cudaStream_t)stream);
    });
    return launched(name, e);
}

extern "C" size_t bq_residual_norm_backward_workspace_bytes(int32_t T, int32_t H) {
    if (T < 0 || H < 8 || H % 8 || H > kMaxH) return 0;
    return (size_t)std::max(1, std::min(T, kMaxBlocks)) * H * 4 * 2;   // a part per block, of two sums
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
    RingMaker ring;
    ring.put(kY, y, ldy, d->y_dtype);
    if (dx) {
        ring.put(kOut, h_out, ldho, d->h_dtype);
        ring.put(kDx, dx, lddx, d->x_dtype);
    }
    if (dh_out) ring.put(kDout, dh_out, lddho, d->h_dtype);
    if (d->gate_kind == BQ_GATE_FULL) ring.put(kFull, d->gate, d->ldgate, d->gate_dtype);
    const Shape p = shape_of(d->T, d->H, ring.bytes);
    if (sums) {
        const size_t need = bq_residual_norm_backward_workspace_bytes(d->T, d->H);
        if (!workspace || workspace_bytes < need)
            return bq::fail(BQ_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu", name, workspace_bytes, need);
        if (!bq::aligned(workspace, 16)) return bq::fail(BQ_ERR_ALIGN, "%s: workspace must be 16-byte aligned", name);
    }
    if ((s = bq::check_arch()) != BQ_OK) return s;
    float* channel_gate = channel ? static_cast<float*>(dgate) : nullptr;
    const int i_gain = dgain ? 0 : -1, i_branch = dpost_gain || channel_gate ? i_gain + 1 : -1;
    const Columns columns = columns_of(d, dx != nullptr);
    const SumArgs sum{static_cast<const float*>(workspace), d->T > 0 ? p.blocks : 0, d->H, dgain, dpost_gain,
                      channel_gate, i_gain, i_branch, columns};
    cudaStream_t st = (cudaStream_t)stream;
    if (d->T > 0) {
        const int32_t x_dtype = dx ? d->x_dtype : d->h_dtype;
        const Rows to_dy = rows(dy, lddy, d->y_dtype), to_dh = rows(dh, lddh, d->h_dtype);
        const Rows to_dgate = rows(dgate, lddgate, d->gate_dtype);
        const int64_t step = (int64_t)p.rows * p.blocks;
        const BackwardArgs a{d->T, d->H, ring.laid_out(p, d->H), to_dy, to_dh, columns, to_dgate, to_dy.ld * step,
                             to_dh.ld * step, d->gate_kind == BQ_GATE_FULL ? to_dgate.ld * step : 0, d->residual_scale,
                             d->eps, static_cast<float*>(workspace), i_gain, i_branch};
        cudaError_t e = cudaSuccess;
        with_types(d->y_dtype, d->h_dtype, x_dtype, [&](auto type) {
            using D = decltype(type);
            if (p.cluster > 1) e = p.per_thread == 1 ? launch_rows<residual_norm_backward_kernel<kAny, kAny, kAny, 1, true>>(p, a, st)
                                              : launch_rows<residual_norm_backward_kernel<kAny, kAny, kAny, 2, true>>(p, a, st);
            else if (p.per_thread == 1) e = launch_rows<residual_norm_backward_kernel<D::y, D::h, D::x, 1, false>>(p, a, st);
            else e = launch_rows<residual_norm_backward_kernel<D::y, D::h, D::x, 2, false>>(p, a, st);
        });
        if ((s = launched(name, e)) != BQ_OK) return s;
    }
    if (!sums) return BQ_OK;
    return launched(name, bq::launch_after(sum_parts_kernel, dim3((d->H + 31) / 32, (i_gain >= 0) + (i_branch >= 0)), dim3(kSumThreads), 0, st,
                                           sum));
}
