// Gradients of the residual norm (resnorm.cu has the formulas).
//
// With P = scale * post_gain * (a gate per channel), f the gate per token and w
// the one per value (or 1 each), yn = s y (y without a post norm):
//   dy = f (s P w G - y s^3 mean(P w G y)), or f P w G;   Q = sum over rows of f w G yn
//   dpost_gain = scale gate Q;   dgate per channel = scale gate' post_gain Q
//   dgate per token = gate' sum of P G yn;   dgate per value = P G yn w'
// so one column sum serves both gradients of the branch, and the constants are
// folded in at the end.  The sum of P w G y is linear in G = dh' + r gain dx - h' c:
// its three parts need neither r nor c, so every sum over a row is formed in one
// pass and one barrier, and a second pass writes all outputs.
//
// Four rows are read and two written (GB300, bf16, post norm, gate per channel:
// 8192 x 4096 72 us, 5.6 TB/s; 2048 x 4096 27 us, 3.7 TB/s).  From 2048 to 8192
// rows a row costs 7.4 ns, at the copy bandwidth 7.2: memory bounds the walk, with
// the 16 warps an SM that 114 to 120 registers leave issuing in half of the cycles.
// 12 us are fixed: 6 are the column sums (without them 21.8 us: 304 parts of two
// sums, 10 MB, are written and read again by a second kernel), the others the
// launch, the first rows on their way and the last ones (2048 rows are 6.7 rounds
// of 304 blocks).  With an fp32 stream and a gate per value (2047 x 2048 24 us) a
// row costs 8.8 ns, at the copy bandwidth 6.6; why was not found.
// Steps that led here, 2048 x 4096: rows fetched ahead
// 85 -> 48 us, packed arithmetic and constants kept as fp32 37, two blocks an SM
// 31, all sums of a row in one barrier 28.
#include "resnorm.cuh"

namespace {

using namespace bq;
using namespace bq::resnorm;

template <int DY, int DH, int DX, int THREADS, int VPT>
struct Stage {
    static constexpr int kPlane = THREADS * VPT * 16;
    static constexpr int kY = 0, kOut = kY + planes(DY) * kPlane, kDx = kOut + planes(DH) * kPlane;
    static constexpr int kDout = kDx + planes(DX) * kPlane, kGate = kDout + planes(DH) * kPlane;   // last
    static constexpr int kGain = 0, kBranch = 2 * kPlane;   // constants, fp32, in front of the stages
};

struct BackwardArgs {
    int T, H, slice;                // slice: vectors of a row in this CTA (a cluster shares a row)
    int stages, stage_bytes, at_stages;   // bytes
    Rows y, out, dout, dx;          // dout.p or dx.p NULL: no gradient comes that way
    Rows dy, dh;
    Columns columns;
    Rows full, dgate;               // a gate per value; dgate of one per token (fp32) or per value, p NULL: not computed
    float residual_scale, eps;
    float* part;                    // [arrays][parts][H] column sums: dgain, Q
    int sum_gain, sum_branch;       // which array each is, or -1
};

// blockDim.x threads take a row (or a cluster's slice of one), a thread the vectors x, x + blockDim.x of it;
// blockDim.y rows at a time.  Blocks walk over the rows; a thread's columns stay the same, so it adds their column sums
// in registers.  Each thread fetches the vectors that it will use itself, rows ahead, into shared memory of its own
// (cp.async): the loads need no registers while they are in flight, and no barrier when they land.  A vector behind the
// row's last, and a row behind the last, is zeros there: the arithmetic goes over all alike.
template <int DY, int DH, int DX, int THREADS, int VPT, bool POST, bool CLUSTER>
__global__ void __launch_bounds__(THREADS, 512 / THREADS)
residual_norm_backward_kernel(const __grid_constant__ BackwardArgs a) {
    using L = Stage<DY, DH, DX, THREADS, VPT>;
    constexpr int PLANE = L::kPlane;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ SumBuf s_buf;
    const Gate& gate = a.columns.gate;
    const bool has_x = a.dx.p != nullptr, full = gate.kind == GATE_FULL;
    const bool branch_kept = POST || gate.kind == GATE_CHANNEL;   // else its constant is scale alone
    const bool token = gate.kind == GATE_TOKEN && a.dgate.p;   // its gradient is wanted
    const int vecs = a.H / 8, tid = threadIdx.y * blockDim.x + threadIdx.x;
    const int ranks = CLUSTER ? (vecs + a.slice - 1) / a.slice : 1, rank = CLUSTER ? (int)cluster_rank() : 0;
    const int mine = min(a.slice, vecs - rank * a.slice), vec0 = rank * a.slice + threadIdx.x;
    bool has[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) has[v] = (int)(threadIdx.x + v * blockDim.x) < mine;
    const int64_t step = (int64_t)(gridDim.x / ranks) * blockDim.y, block0 = (int64_t)(blockIdx.x / ranks) * blockDim.y;
    // a thread's first vector in the rows of a block, from the block's first row on (the host made sure that it is an int)
    auto offset = [&](const Rows& m) { return (int)threadIdx.y * m.ld16 * 16 + vec0 * vec_bytes(m.dtype); };
    const int o_y = offset(a.y), o_out = offset(a.out), o_dx = offset(a.dx), o_dout = offset(a.dout);
    const int o_dy = offset(a.dy), o_dh = offset(a.dh);
    const int end = a.at_stages + a.stages * a.stage_bytes;
    uint8_t* own = smem + tid * 16;
    zero_missing<PLANE>(own, end, has);
    // launched behind whatever precedes it on the stream: nothing before this line touches global memory
    bq::grid_dependency_wait();
    bq::allow_dependents();
    const uint32_t own_u32 = (uint32_t)__cvta_generic_to_shared(own);
    auto fetch_vector = [&](uint32_t to, int64_t r0, int v) {
        fetch_one<DY, PLANE, VPT>(to + L::kY, a.y.row(r0) + o_y, a.y.dtype, v);
        if (has_x) {
            fetch_one<DH, PLANE, VPT>(to + L::kOut, a.out.row(r0) + o_out, a.out.dtype, v);
            fetch_one<DX, PLANE, VPT>(to + L::kDx, a.dx.row(r0) + o_dx, a.dx.dtype, v);
        }
        if (a.dout.p) fetch_one<DH, PLANE, VPT>(to + L::kDout, a.dout.row(r0) + o_dout, a.dout.dtype, v);
        if (full) fetch_one<DY, PLANE, VPT>(to + L::kGate, a.full.row(r0) + offset(a.full), a.full.dtype, v);
    };
    auto fetch_row = [&](int stage, int64_t r0) {
        const uint32_t to = own_u32 + stage;
        if (r0 + threadIdx.y < a.T) {
#pragma unroll
            for (int v = 0; v < VPT; ++v)
                if (has[v]) fetch_vector(to, r0, v);
        } else if (r0 < a.T) {
            for (int i = 0; i < a.stage_bytes; i += PLANE / VPT)
                *reinterpret_cast<uint4*>(own + stage + i) = make_uint4(0, 0, 0, 0);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // With room for one row only (blocks of 512 threads with one row at a time), a vector's place is filled again once the
    // vector has been used for the last time (2048 x 8192 fp32 124 us, 127 with the whole row fetched at its turn; fp32
    // stream between bf16 rows 88 and 92).
    const bool refill = THREADS * VPT == 1024 && a.stages == 1;
    int ahead = a.at_stages;
    int64_t next = block0;
    for (int i = 0; i < max(a.stages - 1, 1); ++i) {
        fetch_row(ahead, next);
        ahead += a.stage_bytes;
        next += step;
    }
    keep_columns<PLANE, POST>(own + L::kGain, branch_kept ? own + L::kBranch : nullptr, a.columns, vec0, has);
    Vec gain_sum[VPT], branch[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) gain_sum[v] = branch[v] = same8(0.f);
    const float inv_h = 1.f / (float)a.H;
    int stage = a.at_stages, turn = 0;
    for (int64_t t0 = block0; t0 < a.T; t0 += step) {
        const int64_t t = t0 + threadIdx.y;
        const bool live = t < a.T;
        if (a.stages < 3) asm volatile("cp.async.wait_group 0;" ::: "memory");
        else asm volatile("cp.async.wait_group 1;" ::: "memory");
        if (!refill) {
            fetch_row(ahead, next);
            ahead = ahead + a.stage_bytes == end ? a.at_stages : ahead + a.stage_bytes;
        }
        const uint8_t* st = own + stage;
        stage = stage + a.stage_bytes == end ? a.at_stages : stage + a.stage_bytes;
        const float f = token_factor(gate, t, live);
        // sums over the row: h'^2, gain dx h', y^2, and P w y times dh', gain dx and h'
        f32x2 hh = both(0.f), dh = both(0.f), yy = both(0.f), in_dout = both(0.f), in_dx = both(0.f), in_h = both(0.f);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            Vec h, q;   // h', gain dx
            if (has_x) {
                h = staged8<DH, PLANE, VPT>(st + L::kOut, v, a.out.dtype);
                const Vec d = staged8<DX, PLANE, VPT>(st + L::kDx, v, a.dx.dtype);
                q = kept8<PLANE, VPT>(own + L::kGain, v);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    q.p[j] = mul2(d.p[j], q.p[j]);
                    hh = fma2(h.p[j], h.p[j], hh);
                    dh = fma2(q.p[j], h.p[j], dh);
                }
            }
            if (!POST && !token) continue;
            const Vec y = staged8<DY, PLANE, VPT>(st + L::kY, v, a.y.dtype);
            Vec p = branch_kept ? kept8<PLANE, VPT>(own + L::kBranch, v) : same8(a.columns.scale);
            if (full) {
                Vec w = staged8<DY, PLANE, VPT>(st + L::kGate, v, a.full.dtype);
                if (gate.sigmoid) w = sigmoid8(w);
#pragma unroll
                for (int j = 0; j < 4; ++j) p.p[j] = mul2(p.p[j], w.p[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                yy = fma2(y.p[j], y.p[j], yy);
                p.p[j] = mul2(p.p[j], y.p[j]);
            }
            if (has_x) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    in_dx = fma2(p.p[j], q.p[j], in_dx);
                    in_h = fma2(p.p[j], h.p[j], in_h);
                }
            }
            if (a.dout.p) {
                const Vec o = staged8<DH, PLANE, VPT>(st + L::kDout, v, a.dout.dtype);
#pragma unroll
                for (int j = 0; j < 4; ++j) in_dout = fma2(p.p[j], o.p[j], in_dout);
            }
        }
        float sums[8] = {sum2(hh), sum2(dh), sum2(yy), sum2(in_dout), sum2(in_dx), sum2(in_h), 0.f, 0.f};
        if (CLUSTER || POST || token) row_sums<CLUSTER>(sums, s_buf, turn, ranks);
        else if (has_x) row_sums(sums[0], sums[1], s_buf, turn);
        // a row behind the last has sums of 0, whose roots would be infinite without eps; cubes of the roots are taken
        // factor by factor, as they leave fp32's range where their products with the sums do not
        const float r = live ? rsqrtf(__fmaf_rn(sums[0], inv_h, a.eps)) : 0.f, c = -r * (r * (r * (sums[1] * inv_h)));
        const float s = !POST ? 1.f : live ? rsqrtf(__fmaf_rn(sums[2], inv_h, a.eps)) : 0.f;
        float inner = sums[3];           // of P w G y
        if (has_x) inner += r * sums[4] + c * sums[5];
        if (token && live && threadIdx.x == 0 && rank == 0)
            reinterpret_cast<float*>(a.dgate.p)[t] = s * inner * (gate.sigmoid ? f * (1.f - f) : 1.f);
        const float fs = f * s, cy = -fs * (s * (s * (inner * inv_h)));
        uint8_t* to_dh = a.dh.row(t0) + o_dh;
        uint8_t* to_dy = a.dy.row(t0) + o_dy;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const bool stored = live && has[v];
            Vec G = a.dout.p ? staged8<DH, PLANE, VPT>(st + L::kDout, v, a.dout.dtype) : same8(0.f);
            if (has_x) {
                const Vec k = kept8<PLANE, VPT>(own + L::kGain, v), h = staged8<DH, PLANE, VPT>(st + L::kOut, v, a.out.dtype);
                const Vec d = staged8<DX, PLANE, VPT>(st + L::kDx, v, a.dx.dtype);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x2 dr = mul2(d.p[j], both(r));
                    gain_sum[v].p[j] = fma2(dr, h.p[j], gain_sum[v].p[j]);
                    G.p[j] = fma2(h.p[j], both(c), fma2(k.p[j], dr, G.p[j]));
                }
            }
            if (stored) {
                Vec o;
#pragma unroll
                for (int j = 0; j < 4; ++j) o.p[j] = mul2(G.p[j], both(a.residual_scale));
                store8<DH>(to_dh, v * blockDim.x, a.dh.dtype, o);
            }
            const Vec p = branch_kept ? kept8<PLANE, VPT>(own + L::kBranch, v) : same8(a.columns.scale);
            const Vec y = staged8<DY, PLANE, VPT>(st + L::kY, v, a.y.dtype);
            if (full) {
                Vec w = staged8<DY, PLANE, VPT>(st + L::kGate, v, a.full.dtype), dw;
#pragma unroll
                for (int j = 0; j < 4; ++j) dw.p[j] = mul2(mul2(G.p[j], p.p[j]), mul2(y.p[j], both(s)));
                if (gate.sigmoid) {
                    w = sigmoid8(w);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        dw.p[j] = mul2(dw.p[j], mul2(w.p[j], fma2(w.p[j], both(-1.f), both(1.f))));
                }
                if (a.dgate.p && stored)
                    store8<DY>(a.dgate.row(t0) + offset(a.dgate), v * blockDim.x, a.dgate.dtype, dw);
#pragma unroll
                for (int j = 0; j < 4; ++j) G.p[j] = mul2(G.p[j], w.p[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                G.p[j] = mul2(G.p[j], both(fs));
                branch[v].p[j] = fma2(G.p[j], y.p[j], branch[v].p[j]);
                G.p[j] = mul2(G.p[j], p.p[j]);
                if (POST) G.p[j] = fma2(y.p[j], both(cy), G.p[j]);
            }
            if (stored) store8<DY>(to_dy, v * blockDim.x, a.dy.dtype, G);
            if (refill && has[v] && next < a.T) fetch_vector(own_u32 + a.at_stages, next, v);   // behind all uses above
        }
        if (refill) asm volatile("cp.async.commit_group;" ::: "memory");
        next += step;
    }
    // The block's column sums, to its part: a block of one row has them in its threads; of several, they are added up in
    // shared memory (the stages and constants are free, and hold more than two sums).
    const int64_t parts = gridDim.x / ranks, part = blockIdx.x / ranks;
    auto part_of = [&](int which) { return reinterpret_cast<uint8_t*>(a.part + (which * parts + part) * a.H); };
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (blockDim.y == 1) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            if (!has[v]) continue;
            if (a.sum_gain >= 0) store8<BQ_DT_F32>(part_of(a.sum_gain), vec0 + v * blockDim.x, 0, gain_sum[v]);
            if (a.sum_branch >= 0) store8<BQ_DT_F32>(part_of(a.sum_branch), vec0 + v * blockDim.x, 0, branch[v]);
        }
    } else if (a.sum_gain >= 0 || a.sum_branch >= 0) {   // blocks of several rows are not clusters
        const int rows = blockDim.y, quads = 2 * vecs;
        float4* s_sum = reinterpret_cast<float4*>(smem);   // [array][row][quads]
        __syncthreads();
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            if (!has[v]) continue;
            const int at = threadIdx.y * vecs + threadIdx.x + v * blockDim.x;
            if (a.sum_gain >= 0) store8<BQ_DT_F32>(smem, at, 0, gain_sum[v]);
            if (a.sum_branch >= 0) store8<BQ_DT_F32>(smem + (int64_t)a.sum_branch * rows * quads * 16, at, 0, branch[v]);
        }
        __syncthreads();
        const int arrays = 1 + max(a.sum_gain, a.sum_branch);
        for (int i = tid; i < arrays * quads; i += blockDim.x * rows) {
            const int k = i >= quads, c = i - k * quads;
            const float4* from = s_sum + k * rows * quads + c;
            float4 sum = from[0];
#pragma unroll 4
            for (int j = 1; j < rows; ++j) {
                const float4 t = from[j * quads];
                sum.x += t.x;
                sum.y += t.y;
                sum.z += t.z;
                sum.w += t.w;
            }
            reinterpret_cast<float4*>(part_of(k))[c] = sum;
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
// Bound by latency: 304 parts of two sums of 4096 columns (10 MB, in the L2) take 3 to 4 us behind the first kernel.
// All 19 parts of a warp in flight at once, or blocks of 1024 threads, took longer.
__global__ void __launch_bounds__(kSumThreads)
sum_parts_kernel(const SumArgs a) {
    constexpr int kWarps = kSumThreads / 32;
    __shared__ float s_red[kWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    const float* part = a.part + (int64_t)blockIdx.y * a.parts * a.H;
    const Gate& gate = a.columns.gate;
    const bool branch = (int)blockIdx.y == a.sum_branch;
    float f = 1.f, post = 1.f, sum = 0.f;
    bq::grid_dependency_wait();   // nothing before this line touches global memory, which earlier kernels may have written
    bq::allow_dependents();
    // the constants, on their way beside the parts: as they are, since a conversion would wait for its load here (few rows
    // 0.4 us more)
    uint32_t raw_gate = 0, raw_post = 0;
    const bool constants = branch && warp == 0 && c < a.H && a.parts;   // without rows the gate and the gains may be missing
    if (constants) {
        if (gate.kind == GATE_CHANNEL) raw_gate = load_raw(gate.p, c, gate.dtype);
        if (a.columns.post) raw_post = load_raw(a.columns.post, c, a.columns.gain_dtype);
    }
    if (c < a.H) {
#pragma unroll 8
        for (int64_t i = warp; i < a.parts; i += kWarps) sum += part[i * a.H + c];
    }
    s_red[warp][lane] = sum;
    __syncthreads();
    if (warp || c >= a.H) return;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) sum += s_red[w][lane];
    if (!branch) {
        a.dgain[c] = sum;
        return;
    }
    float slope = 1.f;
    if (gate.kind == GATE_CHANNEL) f = raw_value(raw_gate, gate.dtype);
    if (a.columns.post) post = raw_value(raw_post, a.columns.gain_dtype);
    if (gate.kind == GATE_CHANNEL && gate.sigmoid) {
        f = sigmoid_f(f);
        slope = f * (1.f - f);
    }
    sum *= a.columns.scale;
    if (a.dpost) a.dpost[c] = a.parts ? sum * f : 0.f;
    if (a.dgate) a.dgate[c] = a.parts ? sum * slope * post : 0.f;
}

// ---------------------------------------------------------------- host side
// How a call's rows are spread: a cluster of CTAs per row, threads per row, rows of a block, rows in flight.
struct Shape {
    int cluster, slice, block, vpt, threads, rows, stages, stage_bytes, at_stages, blocks;   // blocks: clusters in the grid
    size_t smem;
};

constexpr int kMaxBlocks = 3 * kSms;

// n_planes: of a row's vectors in a stage; n_constants: of the constants.
Shape shape_of(int T, int H, int n_planes, int n_constants) {
    Shape p{};
    const int vecs = H / 8;
    auto bytes = [&](int stages) { return (size_t)(n_constants + stages * n_planes) * p.block * p.vpt * 16; };
    auto fit = [&](int ctas) { return (bytes(2) + 2048) * ctas <= kSmemOfSm; };   // two rows of each
    // a block of 512 threads holds up to 1024 vectors of a row (14 planes of 16 KB at most: four of constants, ten of a
    // row); wider rows are shared by a cluster of two
    static_assert(kMaxH / 8 <= 2 * 1024 && 14 * 1024 * 16 <= kSmemOfSm, "");
    p.cluster = vecs > 1024 ? 2 : 1;
    p.slice = (vecs + p.cluster - 1) / p.cluster;
    p.block = p.slice > 512 ? 512 : 256;
    p.vpt = 2;
    // Two vectors a thread share what a row costs a warp beside them (16384 x 2048 bf16 71 us, one a thread 88; 2400 x
    // 512 10.6 and 10.5).  One where that brings a second CTA to the SM (2048 x 1536 fp32 25.2 us against 27.6), where
    // rows are a warp each way (2400 x 256 7.8 against 8.8), and where a block an SM takes all rows (16 x 2048 5.2
    // against 6.5, 300 x 1024 6.0 against 7.4; 600 x 1024 8.1 and 7.5).
    if (p.slice <= 256 && (!fit(2) || p.slice <= 32 || (int64_t)T * p.slice <= kSms * 256)) p.vpt = 1;
    p.threads = ((p.slice + p.vpt - 1) / p.vpt + 31) / 32 * 32;
    p.rows = p.cluster > 1 ? 1 : std::max(1, p.block / p.threads);
    const int per_sm = p.block == 256 && fit(2) ? 2 : 1;   // what the registers allow
    p.stages = (bytes(3) + 2048) * per_sm <= kSmemOfSm ? 3 : bytes(2) <= kSmemOfSm ? 2 : 1;
    p.stage_bytes = n_planes * p.block * p.vpt * 16;
    p.at_stages = n_constants * p.block * p.vpt * 16;
    p.smem = bytes(p.stages);   // room for the block's two column sums too, 64 bytes per vector: six planes at least
    // clusters of one and of two CTAs that this GPU holds at once, with one CTA an SM
    const int held = kSms / p.cluster;
    p.blocks = (int)std::min<int64_t>(held * per_sm, ((int64_t)T + p.rows - 1) / p.rows);
    return p;
}

template <auto kernel>
cudaError_t launch_rows(const Shape& p, const BackwardArgs& a, cudaStream_t st) {
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

template <int DY, int DH, int DX, bool POST>
cudaError_t launch_backward(const Shape& p, const BackwardArgs& a, cudaStream_t st) {
    if (p.cluster > 1) return launch_rows<residual_norm_backward_kernel<DY, DH, DX, 512, 2, POST, true>>(p, a, st);
    if (p.vpt == 1) return launch_rows<residual_norm_backward_kernel<DY, DH, DX, 256, 1, POST, false>>(p, a, st);
    if (p.block == 256) return launch_rows<residual_norm_backward_kernel<DY, DH, DX, 256, 2, POST, false>>(p, a, st);
    return launch_rows<residual_norm_backward_kernel<DY, DH, DX, 512, 2, POST, false>>(p, a, st);
}

}  // namespace

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
    const bool channel = d->gate_kind == BQ_GATE_CHANNEL, full = d->gate_kind == BQ_GATE_FULL;
    if ((dgain && d->T > 0 && !dx) || (dpost_gain && d->T > 0 && !d->post_gain) || (dgate && d->gate_kind == BQ_GATE_NONE))
        return bq::fail(BQ_ERR_NULL, "%s: a gradient is asked for without what it belongs to (dgain: dx, dpost_gain: "
                                     "post_gain, dgate: gate)", name);
    if (!bq::aligned(dgain, 4) || !bq::aligned(dpost_gain, 4) || (!full && !bq::aligned(dgate, 4)))
        return bq::fail(BQ_ERR_ALIGN, "%s: sums must be 4-byte aligned", name);
    const bool sums = dgain || dpost_gain || (dgate && channel);
    if (d->T == 0 && !sums) return BQ_OK;
    if (d->T > 0) {
        const int ys = bq::dtype_size(d->y_dtype), hs = bq::dtype_size(d->h_dtype);
        if (!dx && !dh_out) return bq::fail(BQ_ERR_NULL, "%s: dx and dh_out are both NULL", name);
        if ((s = check_matrix(name, "y", y, d->H, ldy, ys)) != BQ_OK ||
            (dx && (s = check_matrix(name, "h_out", h_out, d->H, ldho, hs)) != BQ_OK) ||
            (dh_out && (s = check_matrix(name, "dh_out", dh_out, d->H, lddho, hs)) != BQ_OK) ||
            (dx && (s = check_matrix(name, "dx", dx, d->H, lddx, bq::dtype_size(d->x_dtype))) != BQ_OK) ||
            (s = check_matrix(name, "dy", dy, d->H, lddy, ys)) != BQ_OK ||
            (s = check_matrix(name, "dh", dh, d->H, lddh, hs)) != BQ_OK)
            return s;
        if (dgate && full &&
            (s = check_matrix(name, "dgate", dgate, d->H, lddgate, bq::dtype_size(d->gate_dtype))) != BQ_OK)
            return s;
    }
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
    cudaStream_t st = (cudaStream_t)stream;
    Shape p{};
    if (d->T > 0) {
        const int32_t x_dtype = dx ? d->x_dtype : d->h_dtype;
        BackwardArgs a{};
        a.T = d->T;
        a.H = d->H;
        a.y = rows(y, ldy, d->y_dtype);
        a.out = rows(dx ? h_out : nullptr, ldho, d->h_dtype);
        a.dout = rows(dh_out, lddho, d->h_dtype);
        a.dx = rows(dx, lddx, x_dtype);
        a.dy = rows(dy, lddy, d->y_dtype);
        a.dh = rows(dh, lddh, d->h_dtype);
        a.columns = columns;
        if (full) a.full = rows(d->gate, d->ldgate, d->gate_dtype);
        a.dgate = rows(dgate, full ? lddgate : 0, full ? d->gate_dtype : BQ_DT_F32);
        a.residual_scale = d->residual_scale;
        a.eps = d->eps;
        a.part = static_cast<float*>(workspace);
        a.sum_gain = i_gain;
        a.sum_branch = i_branch;
        cudaError_t e = cudaSuccess;
        auto go = [&](auto type, auto post) {
            using D = decltype(type);
            constexpr bool POST = decltype(post)::value;
            const int constants = POST || channel ? 4 : 2;
            p = shape_of(d->T, d->H, (full ? 2 : 1) * planes(D::y) + 2 * planes(D::h) + planes(D::x), constants);
            if (p.rows > 1 && std::max({a.y.ld16, a.out.ld16, a.dout.ld16, a.dx.ld16, a.dy.ld16, a.dh.ld16, a.full.ld16,
                                        a.dgate.ld16}) > INT32_MAX / 256) {
                // offsets inside a block's rows are ints: rows that far apart are taken one at a time
                p.rows = 1;
                p.blocks = std::min(d->T, kMaxBlocks);
            }
            a.slice = p.slice;
            a.stages = p.stages;
            a.stage_bytes = p.stage_bytes;
            a.at_stages = p.at_stages;
            e = launch_backward<D::y, D::h, D::x, POST>(p, a, st);
        };
        with_types(d->y_dtype, d->h_dtype, x_dtype, full ? d->gate_dtype : d->y_dtype, [&](auto type) {
            if (d->post_gain) go(type, std::true_type());
            else go(type, std::false_type());
        });
        if ((s = launched(name, e)) != BQ_OK) return s;
    }
    if (!sums) return BQ_OK;
    const SumArgs sum{static_cast<const float*>(workspace), p.blocks, d->H, dgain, dpost_gain, channel_gate, i_gain, i_branch,
                      columns};
    return launched(name, bq::launch_after(sum_parts_kernel, dim3((d->H + 31) / 32, (i_gain >= 0) + (i_branch >= 0)),
                                           dim3(kSumThreads), 0, st, sum));
}
