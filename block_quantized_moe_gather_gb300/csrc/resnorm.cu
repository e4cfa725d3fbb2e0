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
#include "resnorm.cuh"

namespace {

using namespace bq;
using namespace bq::resnorm;

struct ForwardArgs {
    int T, H;
    Rows y, h, out, x;              // x.p NULL: not computed
    const uint8_t* full;            // a gate per value, and its rows
    int64_t ld_full;
    Columns columns;
    float residual_scale, eps;
};

constexpr int kMaxThreads = 512;

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
    const uint8_t *y = a.y.p + t * a.y.ld, *h = a.h.p + t * a.h.ld;
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
            Vec w = load8<kAny>(gate.kind == GATE_FULL ? a.full + t * a.ld_full : gate.p, i, gate.dtype);
            if (gate.sigmoid) w = sigmoid8(w);
#pragma unroll
            for (int j = 0; j < 4; ++j) r[v].p[j] = mul2(r[v].p[j], w.p[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r[v].p[j] = fma2(r[v].p[j], both(f), mul2(o[v].p[j], both(a.residual_scale)));
            squares = fma2(r[v].p[j], r[v].p[j], squares);
        }
        store8<DH>(a.out.p + t * a.out.ld, i, a.out.dtype, r[v]);
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
        store8<DX>(a.x.p + t * a.x.ld, i, a.x.dtype, r[v]);
    }
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
                        rows(x, ldx, x_dtype), static_cast<const uint8_t*>(d->gate),
                        d->ldgate * bq::dtype_size(d->gate_dtype), columns_of(d, x != nullptr), d->residual_scale, d->eps};
    // Threads of a row: for few rows a vector each, as far as 512 threads go; for many two, so that what a row costs a
    // warp beside its vectors is shared.
    const int vecs = d->H / 8;
    const int per = vecs > 2 * kMaxThreads ? 4 : vecs > kMaxThreads || d->T > kSms ? 2 : 1;
    const int threads = ((vecs + per - 1) / per + 31) / 32 * 32, per_cta = std::max(1, 256 / threads);
    const dim3 grid((unsigned)(((int64_t)d->T + per_cta - 1) / per_cta)), block(threads, per_cta);
    cudaError_t e = cudaSuccess;
    with_types(d->y_dtype, d->h_dtype, x_dtype, [&](auto type) {
        using D = decltype(type);
        auto go = [&](auto kernel) { e = bq::launch_after(kernel, grid, block, 0, (cudaStream_t)stream, a); };
        if (d->post_gain) {
            if (per == 1) go(residual_norm_kernel<D::y, D::h, D::x, 1, true>);
            else if (per == 2) go(residual_norm_kernel<D::y, D::h, D::x, 2, true>);
            else go(residual_norm_kernel<kAny, kAny, kAny, 4, true>);
        } else {
            if (per == 1) go(residual_norm_kernel<D::y, D::h, D::x, 1, false>);
            else if (per == 2) go(residual_norm_kernel<D::y, D::h, D::x, 2, false>);
            else go(residual_norm_kernel<kAny, kAny, kAny, 4, false>);
        }
    });
    return launched(name, e);
}
