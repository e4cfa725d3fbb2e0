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
//
// Every value of y and h is read once and every value of h' and x written once; with many rows that is what bounds the
// pass (GB300, bf16, post norm, gate per channel: 8192 x 4096 44 us, 6.1 TB/s; 2048 x 4096 15.3 us, 4.4 TB/s, of which
// about 4 us are the start and the last rows).  A row has two sums that depend on one another (y^2, then h'^2), so rows
// loaded when their turn comes leave the memory idle in between: where rows outnumber what the SMs hold at once, blocks
// fetch theirs ahead.  Few rows are bound by the latency of one (1 x 4096 2.1 us).
#include "resnorm.cuh"

namespace {

using namespace bq;
using namespace bq::resnorm;

struct ForwardArgs {
    int T, H;
    Rows y, h, out, x;              // x.p NULL: not computed
    Rows full;                      // a gate per value
    Columns columns;
    float residual_scale, eps;
};

constexpr int kMaxThreads = 1024;
constexpr int kThreadsOfGpu = 1024 * kSms;   // of residual_norm_kernel that fit at once: 64 registers each

// blockDim.x threads take a row, a thread the vectors x, x + blockDim.x, ... of it; blockDim.y rows a CTA.
template <int DY, int DH, int DX, int VPT, bool POST>
__global__ void __launch_bounds__(kMaxThreads)
residual_norm_kernel(const __grid_constant__ ForwardArgs a) {
    __shared__ SumBuf s_buf;
    bq::grid_dependency_wait();   // launched behind whatever precedes it on the stream
    bq::allow_dependents();
    const Gate& gate = a.columns.gate;
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int vecs = a.H / 8;
    bool has[VPT];
    Vec r[VPT], o[VPT];
    const uint8_t *y = a.y.row(t), *h = a.h.row(t);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int i = threadIdx.x + v * blockDim.x;
        has[v] = t < a.T && i < vecs;
        r[v] = has[v] ? load8<DY>(y, i, a.y.dtype) : same8(0.f);
        o[v] = has[v] ? load8<DH>(h, i, a.h.dtype) : same8(0.f);
    }
    float f = a.columns.scale * token_factor(gate, t, t < a.T);
    int turn = 0;
    const float inv_h = 1.f / (float)a.H;
    if (POST) {
        f32x2 squares = both(0.f);
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
            for (int j = 0; j < 4; ++j) squares = fma2(r[v].p[j], r[v].p[j], squares);
        f *= rsqrtf(__fmaf_rn(row_sum(sum2(squares), s_buf, turn), inv_h, a.eps));
    }
    f32x2 squares = both(0.f);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int i = threadIdx.x + v * blockDim.x;
        if (!has[v]) continue;
        if (POST) {
            const Vec p = load8<kAny>(a.columns.post, i, a.columns.gain_dtype);
#pragma unroll
            for (int j = 0; j < 4; ++j) r[v].p[j] = mul2(r[v].p[j], p.p[j]);
        }
        if (gate.kind >= GATE_CHANNEL) {
            Vec w = load8<kAny>(gate.kind == GATE_FULL ? a.full.row(t) : gate.p, i, gate.dtype);
            if (gate.sigmoid) w = sigmoid8(w);
#pragma unroll
            for (int j = 0; j < 4; ++j) r[v].p[j] = mul2(r[v].p[j], w.p[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r[v].p[j] = fma2(r[v].p[j], both(f), mul2(o[v].p[j], both(a.residual_scale)));
            squares = fma2(r[v].p[j], r[v].p[j], squares);
        }
        store8<DH>(a.out.row(t), i, a.out.dtype, r[v]);
    }
    if (!a.x.p) return;
    const float norm = rsqrtf(__fmaf_rn(row_sum(sum2(squares), s_buf, turn), inv_h, a.eps));
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int i = threadIdx.x + v * blockDim.x;
        if (!has[v]) continue;
        const Vec c = load8<kAny>(a.columns.gain, i, a.columns.gain_dtype);
#pragma unroll
        for (int j = 0; j < 4; ++j) r[v].p[j] = mul2(mul2(r[v].p[j], both(norm)), c.p[j]);
        store8<DX>(a.x.row(t), i, a.x.dtype, r[v]);
    }
}

// The same for many rows (a vector behind a row's last is zeros): blocks walk over them with the next rows on their way
// (resnorm.cuh) and the columns' constants kept as fp32, so that the loads' latency and the conversions of the gains are
// not paid row by row.  2048 x 4096 bf16: 14.4 us (rows loaded directly 16.2); it issues in half of the cycles, at 24
// warps an SM.
struct ManyArgs {
    ForwardArgs f;
    int stages, stage_bytes, at_stages, at_branch;   // bytes; at_branch -1: the branch's constant is scale alone
};

template <int DY, int DH, int DX, int THREADS, int VPT, bool POST>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
residual_norm_many_kernel(const __grid_constant__ ManyArgs m) {
    constexpr int PLANE = THREADS * VPT * 16;
    constexpr int kY = 0, kH = planes(DY) * PLANE, kFull = kH + planes(DH) * PLANE;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ SumBuf s_buf;
    const ForwardArgs& a = m.f;
    const Gate& gate = a.columns.gate;
    const bool full = gate.kind == GATE_FULL;
    const int vecs = a.H / 8, tid = threadIdx.y * blockDim.x + threadIdx.x;
    bool has[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) has[v] = (int)(threadIdx.x + v * blockDim.x) < vecs;
    const int64_t step = (int64_t)gridDim.x * blockDim.y, block0 = (int64_t)blockIdx.x * blockDim.y;
    const int end = m.at_stages + m.stages * m.stage_bytes;
    uint8_t* own = smem + tid * 16;
    zero_missing<PLANE>(own, end, has);
    const uint32_t own_u32 = (uint32_t)__cvta_generic_to_shared(own);
    // a thread's first vector in the rows of a block, from the block's first row on (the host made sure that it is an int)
    auto offset = [&](const Rows& r) { return (int)threadIdx.y * r.ld16 * 16 + (int)threadIdx.x * vec_bytes(r.dtype); };
    const int o_y = offset(a.y), o_h = offset(a.h), o_full = offset(a.full), o_out = offset(a.out), o_x = offset(a.x);
    // launched behind whatever precedes it on the stream: nothing before this line touches global memory
    bq::grid_dependency_wait();
    bq::allow_dependents();
    auto fetch_row = [&](int stage, int64_t r0) {
        const uint32_t to = own_u32 + stage;
        if (r0 + threadIdx.y < a.T) {
            fetch<DY, PLANE>(to + kY, a.y.row(r0) + o_y, a.y.dtype, has);
            fetch<DH, PLANE>(to + kH, a.h.row(r0) + o_h, a.h.dtype, has);
            if (full) fetch<DY, PLANE>(to + kFull, a.full.row(r0) + o_full, gate.dtype, has);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int ahead = m.at_stages;
    int64_t next = block0;
    for (int i = 0; i < m.stages - 1; ++i) {
        fetch_row(ahead, next);
        ahead += m.stage_bytes;
        next += step;
    }
    const bool branch = m.at_branch >= 0;
    keep_columns<PLANE, POST>(own, branch ? own + m.at_branch : nullptr, a.columns, threadIdx.x, has);
    const float inv_h = 1.f / (float)a.H;
    int stage = m.at_stages, turn = 0;
    for (int64_t t0 = block0; t0 < a.T; t0 += step) {
        const int64_t t = t0 + threadIdx.y;
        const bool live = t < a.T;
        if (m.stages == 2) asm volatile("cp.async.wait_group 0;" ::: "memory");
        else asm volatile("cp.async.wait_group 1;" ::: "memory");
        fetch_row(ahead, next);
        next += step;
        ahead = ahead + m.stage_bytes == end ? m.at_stages : ahead + m.stage_bytes;
        const uint8_t* st = own + stage;
        stage = stage + m.stage_bytes == end ? m.at_stages : stage + m.stage_bytes;
        float f = token_factor(gate, t, live);
        if (!branch) f *= a.columns.scale;
        Vec r[VPT];
#pragma unroll
        for (int v = 0; v < VPT; ++v) r[v] = staged8<DY, PLANE, VPT>(st + kY, v, a.y.dtype);
        if (POST) {
            f32x2 squares = both(0.f);
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int j = 0; j < 4; ++j) squares = fma2(r[v].p[j], r[v].p[j], squares);
            f *= rsqrtf(__fmaf_rn(row_sum(sum2(squares), s_buf, turn), inv_h, a.eps));
        }
        f32x2 squares = both(0.f);
        uint8_t* to_out = a.out.row(t0) + o_out;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const Vec o = staged8<DH, PLANE, VPT>(st + kH, v, a.h.dtype);
            if (branch) {
                const Vec c = kept8<PLANE, VPT>(own + m.at_branch, v);
#pragma unroll
                for (int j = 0; j < 4; ++j) r[v].p[j] = mul2(r[v].p[j], c.p[j]);
            }
            if (full) {
                Vec w = staged8<DY, PLANE, VPT>(st + kFull, v, gate.dtype);
                if (gate.sigmoid) w = sigmoid8(w);
#pragma unroll
                for (int j = 0; j < 4; ++j) r[v].p[j] = mul2(r[v].p[j], w.p[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                r[v].p[j] = fma2(r[v].p[j], both(f), mul2(o.p[j], both(a.residual_scale)));
                squares = fma2(r[v].p[j], r[v].p[j], squares);
            }
            if (live && has[v]) store8<DH>(to_out, v * blockDim.x, a.out.dtype, r[v]);
        }
        if (!a.x.p) continue;
        const float norm = rsqrtf(__fmaf_rn(row_sum(sum2(squares), s_buf, turn), inv_h, a.eps));
        uint8_t* to_x = a.x.row(t0) + o_x;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const Vec c = kept8<PLANE, VPT>(own, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) r[v].p[j] = mul2(mul2(r[v].p[j], both(norm)), c.p[j]);
            if (live && has[v]) store8<DX>(to_x, v * blockDim.x, a.x.dtype, r[v]);
        }
    }
}

// Blocks that would take more than this leave an SM one row ahead of one row; there rows loaded directly, two blocks an
// SM, are faster (2048 x 8192 fp32 with a post norm and a gate per channel, 192 KB: 56 us against 71; fp32 stream between
// bf16 rows 44 against 47).
constexpr size_t kManySmem = 150 * 1024;

template <auto kernel>
cudaError_t launch_many(const ManyArgs& m, dim3 grid, dim3 block, size_t smem, cudaStream_t st) {
    // per device: the attribute is a property of the function on the current device
    static std::atomic<bool> attr_set[64];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_set[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemOfSm);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(true, std::memory_order_release);
    }
    return bq::launch_after(kernel, grid, block, smem, st, m);
}

}  // namespace

extern "C" bq_status bq_residual_norm(const bq_residual_norm_desc* d, const void* y, int64_t ldy, const void* h,
                                      int64_t ldh, void* h_out, int64_t ldho, void* x, int64_t ldx,
                                      bq_stream_t stream) {
    const char* name = "bq_residual_norm";
    bq_status s = check_desc(name, d, x != nullptr);
    if (s != BQ_OK || d->T == 0) return s;
    const int ys = bq::dtype_size(d->y_dtype), hs = bq::dtype_size(d->h_dtype);
    if ((s = check_matrix(name, "y", y, d->H, ldy, ys)) != BQ_OK ||
        (s = check_matrix(name, "h", h, d->H, ldh, hs)) != BQ_OK ||
        (s = check_matrix(name, "h_out", h_out, d->H, ldho, hs)) != BQ_OK)
        return s;
    if (x && (s = check_matrix(name, "x", x, d->H, ldx, bq::dtype_size(d->x_dtype))) != BQ_OK) return s;
    if ((s = bq::check_arch()) != BQ_OK) return s;
    const int32_t x_dtype = x ? d->x_dtype : d->h_dtype;
    const bool full_gate = d->gate_kind == BQ_GATE_FULL;
    const int32_t full_dtype = full_gate ? d->gate_dtype : d->y_dtype;
    const ForwardArgs a{d->T, d->H, rows(y, ldy, d->y_dtype), rows(h, ldh, d->h_dtype), rows(h_out, ldho, d->h_dtype),
                        rows(x, ldx, x_dtype), full_gate ? rows(d->gate, d->ldgate, d->gate_dtype) : Rows{},
                        columns_of(d, x != nullptr), d->residual_scale, d->eps};
    // Threads of a row: a vector each while all rows are on the SMs at once that way (200 x 2048 2.8 us against 3.4 with
    // two, 200 x 4096 3.4 against 3.7; 600 x 4096 8.7 against 6.0); rows of one warp leave it no fewer threads with two
    // (4000 x 256 3.3 us with one, 2.8 with two).
    const int vecs = d->H / 8;
    const int64_t all_vecs = (int64_t)d->T * vecs;
    const int per = vecs > 512 || vecs <= 32 || all_vecs > kThreadsOfGpu ? 2 : 1;
    const int threads = ((vecs + per - 1) / per + 31) / 32 * 32, per_cta = std::max(1, 256 / threads);
    const dim3 grid((unsigned)(((int64_t)d->T + per_cta - 1) / per_cta)), block(threads, per_cta);
    cudaError_t e = cudaSuccess;
    bool done = false;
    // More rows than the SMs hold at once with two vectors a thread, of which a block of 256 or 512 threads holds one or
    // more; two vectors a thread where one does not do.  (600 x 4096: 7.6 us this way, 6.0 loaded directly; 1216 x 2048
    // 6.9 and 6.1; 912 x 4096 8.5 and 9.8; 1824 x 2048 8.7 and 9.9; 2048 x 4096 14.4 and 16.2.)
    const int wide_block = vecs > 512 ? 512 : 256, vpt = vecs > 256 ? 2 : 1;
    const int far = std::max({a.y.ld16, a.h.ld16, a.out.ld16, a.x.ld16, a.full.ld16});
    if (all_vecs > 2 * kThreadsOfGpu && vecs <= 1024 && far <= INT32_MAX / 256) {   // offsets inside a block's rows are ints
        with_types(d->y_dtype, d->h_dtype, x_dtype, full_dtype, [&](auto type) {
            using D = decltype(type);
            const bool branch = d->post_gain || d->gate_kind == BQ_GATE_CHANNEL;
            const int plane = wide_block * vpt * 16, full = full_gate ? planes(D::y) : 0;
            ManyArgs m{a, 2, (planes(D::y) + planes(D::h) + full) * plane, (branch ? 4 : 2) * plane, branch ? 2 * plane : -1};
            auto smem = [&] { return (size_t)m.at_stages + (size_t)m.stages * m.stage_bytes; };
            if (smem() > kManySmem) return;
            done = true;
            const int per_sm = (int)std::max<size_t>(1, std::min<size_t>(1024 / wide_block, kSmemOfSm / (smem() + 2048)));
            if (smem() + m.stage_bytes + 2048 <= kSmemOfSm / per_sm) m.stages = 3;
            const int x_threads = ((vecs + vpt - 1) / vpt + 31) / 32 * 32, row_groups = std::max(1, wide_block / x_threads);
            const int64_t blocks = std::min<int64_t>(kSms * per_sm, ((int64_t)d->T + row_groups - 1) / row_groups);
            const dim3 g((unsigned)blocks), b(x_threads, row_groups);
            cudaStream_t st = (cudaStream_t)stream;
            auto go = [&](auto post) {
                constexpr bool POST = decltype(post)::value;
                if (vpt == 1) e = launch_many<residual_norm_many_kernel<D::y, D::h, D::x, 256, 1, POST>>(m, g, b, smem(), st);
                else if (wide_block == 256)
                    e = launch_many<residual_norm_many_kernel<D::y, D::h, D::x, 256, 2, POST>>(m, g, b, smem(), st);
                else e = launch_many<residual_norm_many_kernel<D::y, D::h, D::x, 512, 2, POST>>(m, g, b, smem(), st);
            };
            if (d->post_gain) go(std::true_type());
            else go(std::false_type());
        });
        if (done) return launched(name, e);
    }
    with_types(d->y_dtype, d->h_dtype, x_dtype, full_dtype, [&](auto type) {
        using D = decltype(type);
        auto go = [&](auto kernel) { e = bq::launch_after(kernel, grid, block, 0, (cudaStream_t)stream, a); };
        if (d->post_gain) {
            if (per == 1) go(residual_norm_kernel<D::y, D::h, D::x, 1, true>);
            else go(residual_norm_kernel<D::y, D::h, D::x, 2, true>);
        } else {
            if (per == 1) go(residual_norm_kernel<D::y, D::h, D::x, 1, false>);
            else go(residual_norm_kernel<D::y, D::h, D::x, 2, false>);
        }
    });
    return launched(name, e);
}
