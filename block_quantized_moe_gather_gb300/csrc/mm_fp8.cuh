// Products of FP8 rows (one scale per 128 values) with FP8 weights (one scale
// per 128 x 128 block), for one weight and for rows sorted by expert.
//
//   y[r][c] = sum_b xs[r][b] ws[c/128][b] * sum_{i in block b} x[r][i] w[c][i]
//
// The sum over one block of 128 is a tcgen05 product of e4m3 operands into
// fp32 TMEM columns (K = 128 = four MMAs of 32).  The scales differ from block
// to block and are not powers of two, so they cannot be part of the MMA: every
// block gets TMEM columns of its own from a ring, and the epilogue warps read
// it and add it, scaled, to fp32 sums in registers while the tensor cores work
// on the next blocks.
#pragma once

#include <algorithm>
#include <atomic>

#include "gemm_internal.cuh"
#include "packed_f32.cuh"
#include "row_chunks.cuh"
#include "row_types.cuh"
#include "tc_ptx.cuh"

namespace bq {
namespace fp8mm {

using namespace bq::tc;

constexpr int kBlock = 128;        // K per scale, per TMA box (one 128-byte swizzle row) and per TMEM stage
constexpr int kMaxExperts = 1024;
constexpr int kMaxCluster = 8;
constexpr int kMaxSize = INT32_MAX - 255;   // of rows, n and k: the row or column behind the last tile is still an int

struct Args {
    const float* xs;
    int rows;
    const int32_t* offsets;   // [E + 1], or NULL: all rows take matrix 0
    int E;
    const float* ws;
    int n, k, kb, nb;         // kb, nb: blocks along k and n
    int cols;                 // columns of y: n, or n/2 with SwiGLU
    void* y;
    int ydtype;
    int64_t ldy;
    int32_t* status;
    unsigned long long wait_limit_ns;
    int skip_copies;          // test only: the producer issues no copies (waits run out); 3: only in a part of a cluster
    int max_chunks;           // row chunks that offsets in order can make
};

// Of kernels with an end: y = scale * act(product + bias) + residual.  Those without take Args alone: with these fields
// behind it, unused, the wide kernel with SwiGLU spilled 24 bytes of its sums a thread instead of 4.
struct EndArgs : Args {
    const float* bias;        // [E][n], or NULL
    int act;                  // bq_activation
    float scale;
    const void* residual;     // rows like y's, or NULL
    int64_t ldr;
};

template <bool END>
using ArgsOf = std::conditional_t<END, EndArgs, Args>;

// ---------------------------------------------------------------- PTX used here only
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar) : "memory");
}

__device__ __forceinline__ void copy4_async(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// The barrier gets this thread's arrival once its copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// kind::f8f6f4, e4m3 (format 0) A and B, fp32 D, both K-major, M = 128, N = n:
// the same fields as the fp16 descriptor.
__device__ __forceinline__ uint32_t idesc_e4m3(int n) { return idesc_f16(n); }

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}

// One lane of a converged warp.  A warp that runs its loop as a whole and lets one lane issue keeps addresses and
// descriptors in uniform registers, which the MMA and TMA instructions take them from.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}

// Bounded wait of a converged warp for a phase of each of two barriers, tested together (one test latency instead of
// two); false if the CTA is aborting or the wait ran out.
__device__ __forceinline__ bool warp_wait_both(uint32_t bar0, uint32_t parity0, uint32_t bar1, uint32_t parity1,
                                               volatile uint32_t* abort_flag, int32_t* status,
                                               unsigned long long limit_ns) {
    unsigned long long t0 = 0;
    for (int i = 1;; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p, q;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
            " mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n and.pred p, p, q;\n selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok) : "r"(bar0), "r"(parity0), "r"(bar1), "r"(parity1) : "memory");
        if (__all_sync(0xffffffffu, ok != 0)) return true;
        if (i % 32 == 0) {
            if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
            const unsigned long long t = __shfl_sync(0xffffffffu, global_ns(), 0);
            if (t0 == 0) t0 = t;
            if (t - t0 > limit_ns) {
                *abort_flag = 1u;
                bq::set_device_error(status, BQ_DEV_WAIT_TIMEOUT);
                return false;
            }
        }
    }
}

// Waits for this warp's TMEM loads; the values pass through so that no use of them moves before the wait.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                   "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                   "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
                 ::"memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ float peer_load(uint32_t addr, uint32_t rank) {
    float v;
    asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %1, %2;\n ld.shared::cluster.f32 %0, [a];\n}\n"
                 : "=f"(v) : "r"(addr), "r"(rank));
    return v;
}

__device__ __forceinline__ uint32_t peer_load_u32(uint32_t addr, uint32_t rank) {
    uint32_t v;
    asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %1, %2;\n ld.shared::cluster.u32 %0, [a];\n}\n"
                 : "=r"(v) : "r"(addr), "r"(rank));
    return v;
}

__device__ __forceinline__ float silu_f(float g) { return __fdividef(g, 1.f + expf(-g)); }

// A load that stays where it is written (the compiler would move it to its use, a block later, and wait there).
__device__ __forceinline__ float load_early(const float* p) {
    float v;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

// ---------------------------------------------------------------- ends
// The activations of the products' ends.  Two special-function instructions each (exp2, reciprocal) bound them, 2.1 us
// for a tile of 128 x 256; what else they take is kept to less than that.  Both are off by 2 units in the last place at
// most; results below the normal range become 0.  No MMA runs meanwhile, as the warps that end a tile are those that
// scale the blocks of the next.  2048 x 4096 x 4096, bf16 out (two tiles a CTA): 30.9 us without an end, bias 32.1, relu
// and bias 32.9, silu 36.1, gelu 37.0; bias and residual, whose rows cost 2.3 us a tile, 36.3.
__device__ __forceinline__ float exp2_approx(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float rcp_approx(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

constexpr float kLog2E = 1.4426950408889634f;

__device__ __forceinline__ float silu_end(float v) { return v * rcp_approx(1.f + exp2_approx(-kLog2E * v)); }

__device__ __forceinline__ float gelu_tanh_end(float v) {   // (1 + tanh(u)) / 2 is sigmoid(2 u)
    const float u = __fmaf_rn(0.044715f * v * v, v, v);
    return v * rcp_approx(1.f + exp2_approx(-kLog2E * 1.5957691216057308f * u));
}

// Two gelus, v Phi(v).  The normal distribution's tail is Phi(-|v|) = exp(-v^2 / 2) R(|v|) with R(a) = erfcx(a / sqrt(2)) / 2,
// which falls from 1/2 like 1 / a: R = t Q(t), t = 1 / (1 + 0.3125 a), Q a polynomial of degree 7 fitted to it on [0, 14.5]
// (largest relative error 2e-7; 5e-7 evaluated in fp32).  The exponent's argument adds v^2 2^-23 at most.  The value is
// max(v, 0) - a Phi(-a) with a = min(|v|, 16), behind which the tail is 0 in fp32 (so that -inf gives 0): it keeps its
// relative precision where it is small.  (An absolute fit of erfc with selects in place of the maximum, off by 5e-4 of the
// value at v = -4, took 38.4 us for the product above.)
__device__ __forceinline__ float max0_or_nan(float v) {
    float r;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ void gelu_end(float& v0, float& v1) {
    const f32x2 a = two(fmaxf(-fabsf(v0), -16.f), fmaxf(-fabsf(v1), -16.f));   // negative
    const float2 den = parts_of(fma2(a, both(-0.3125f), both(1.f)));
    const f32x2 t = two(rcp_approx(den.x), rcp_approx(den.y));
    f32x2 q = fma2(t, both(0.03512295606f), both(-0.1349757326f));
    q = fma2(t, q, both(0.1389943305f));
    q = fma2(t, q, both(-0.003339469029f));
    q = fma2(t, q, both(0.1048217568f));
    q = fma2(t, q, both(0.1098319998f));
    q = fma2(t, q, both(0.1248806164f));
    q = fma2(t, q, both(0.1246636379f));
    const float2 e = parts_of(mul2(mul2(a, both(-0.5f * kLog2E)), a));
    const f32x2 tail = mul2(mul2(q, t), two(exp2_approx(e.x), exp2_approx(e.y)));
    const float2 y = parts_of(fma2(a, tail, two(max0_or_nan(v0), max0_or_nan(v1))));
    v0 = y.x;
    v1 = y.y;
}

// What a kernel with an end is compiled for: the code of every activation in one kernel (and of the residual) cost a
// prefill tile 1.6 us even where none of it ran.
enum { END_NONE = 0, END_SIMPLE, END_SILU, END_GELU, END_GELU_TANH, END_ANY };   // simple: none, relu, relu2, and SwiGLU

// Activations other than SwiGLU, in place: those that END names.  The branch is the same for every thread, and outside
// the values' loop: the code of one activation lies together.
template <int END, int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
    static_assert(N % 2 == 0, "");
    auto all = [&](auto f) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = f(v[i]);
    };
    auto gelu = [&] {
#pragma unroll
        for (int i = 0; i < N; i += 2) gelu_end(v[i], v[i + 1]);
    };
    if (END == END_SILU) {
        all([](float x) { return silu_end(x); });
    } else if (END == END_GELU) {
        gelu();
    } else if (END == END_GELU_TANH) {
        all([](float x) { return gelu_tanh_end(x); });
    } else if (act == BQ_ACT_RELU) {
        all([](float x) { return x < 0.f ? 0.f : x; });
    } else if (act == BQ_ACT_RELU2) {
        all([](float x) { return x < 0.f ? 0.f : x * x; });
    } else if (END == END_ANY) {
        if (act == BQ_ACT_SILU) all([](float x) { return silu_end(x); });
        else if (act == BQ_ACT_GELU) gelu();
        else if (act == BQ_ACT_GELU_TANH) all([](float x) { return gelu_tanh_end(x); });
    }
}

// Element i of a matrix of y's type.
__device__ __forceinline__ float load_value(const void* p, int64_t i, int dtype) {
    if (dtype == BQ_DT_F32) return static_cast<const float*>(p)[i];
    if (dtype == BQ_DT_F16) return __half2float(static_cast<const __half*>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// Column c of rows row0, row0 + step, ... of the residual, those below `end`; 0 where there is none.  The branch on the
// type is outside the loop, so that the loads are in flight together (inside it they came one after the other, 1.5 us
// for 8 rows).
template <int N>
__device__ __forceinline__ void load_residual(const EndArgs& a, int64_t row0, int step, int64_t end, int c, float (&r)[N]) {
    uint32_t raw[N];
#pragma unroll
    for (int i = 0; i < N; ++i) raw[i] = 0;
    if (!a.residual || c >= a.cols) {
    } else if (a.ydtype == BQ_DT_F32) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (row0 + (int64_t)i * step < end)
                raw[i] = static_cast<const uint32_t*>(a.residual)[(row0 + (int64_t)i * step) * a.ldr + c];
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (row0 + (int64_t)i * step < end)
                raw[i] = static_cast<const uint16_t*>(a.residual)[(row0 + (int64_t)i * step) * a.ldr + c];
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        r[i] = a.ydtype == BQ_DT_F32   ? __uint_as_float(raw[i])
               : a.ydtype == BQ_DT_F16 ? __half2float(__ushort_as_half((unsigned short)raw[i]))
                                       : __uint_as_float(raw[i] << 16);
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Lines of a row of the residual, columns [c, c + cols) (bounded), on their way into the L2.
__device__ __forceinline__ void prefetch_residual(const EndArgs& a, int64_t row, int c, int cols) {
    const int es = a.ydtype == BQ_DT_F32 ? 4 : 2, end = min(c + cols, a.cols);
    const uint8_t* p = static_cast<const uint8_t*>(a.residual) + (row * a.ldr + c) * es;
    for (int i = 0; i < (end - c) * es; i += 128) prefetch_l2(p + i);
}

// ---------------------------------------------------------------- work items
// The row chunks of an expert of rows [lo, hi): a chunk is at most `most`
// rows, an expert's rows are cut into chunks of near-equal size.
__device__ __forceinline__ int chunks_of(const Args& a, int lo, int hi, int most) {
    if (!(0 <= lo && lo <= hi && hi <= a.rows)) {
        bq::set_device_error(a.status, BQ_DEV_BAD_ROW);
        return 0;
    }
    return bq::row_chunks(hi - lo, most);
}

// What the CTA keeps of it in shared memory.
struct Chunks {
    int32_t before[kMaxExperts + 1];   // [e]: chunks of the experts before e, [E]: of all that are computed
    int32_t first[kMaxExperts + 1];    // [e]: first row of expert e, [E]: end of the last
    int32_t pad[2];                    // to a multiple of 16 bytes
};
static_assert(sizeof(Chunks) % 16 == 0, "what lies behind it is 16-byte aligned");

// Fills it (all threads of the CTA; ends with a barrier).  Ranges that overlap
// (so descending offsets) can hold more chunks than max_chunks, up to 2^36:
// the sums stop one above max_chunks, and the first expert that passes it and
// all behind it are left out ([E] counts the experts before them).
__device__ __forceinline__ void count_chunks(const Args& a, int most, Chunks* ch) {
    if (!a.offsets) {
        if (threadIdx.x == 0) {
            ch->before[0] = ch->first[0] = 0;
            ch->before[1] = bq::row_chunks(a.rows, most);
            ch->first[1] = a.rows;
        }
    } else if (threadIdx.x < 32) {
        // one warp, four experts a lane
        int total = 0, used = 0;
        for (int e0 = 4 * (int)threadIdx.x; e0 - 4 * (int)threadIdx.x < a.E; e0 += 128) {
            int offset[5], c[4], incl = 0;
#pragma unroll
            for (int i = 0; i < 5; ++i) offset[i] = __ldg(a.offsets + min(e0 + i, a.E));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c[i] = e0 + i < a.E ? chunks_of(a, offset[i], offset[i + 1], most) : 0;
                incl = bq::add_chunks(incl, c[i], a.max_chunks);
            }
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, off);
                if ((int)threadIdx.x >= off) incl = bq::add_chunks(incl, v, a.max_chunks);
            }
            const int behind = __shfl_up_sync(0xffffffffu, incl, 1);
            int before = threadIdx.x ? bq::add_chunks(total, behind, a.max_chunks) : total;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (e0 + i < a.E) {
                    ch->first[e0 + i] = offset[i];
                    ch->before[e0 + i] = before;
                }
                before = bq::add_chunks(before, c[i], a.max_chunks);
                if (before <= a.max_chunks) used = before;   // the sums ascend
            }
            total = bq::add_chunks(total, __shfl_sync(0xffffffffu, incl, 31), a.max_chunks);
        }
        used = __reduce_max_sync(0xffffffffu, used);
        if (threadIdx.x == 0) {
            ch->before[a.E] = used;
            ch->first[a.E] = __ldg(a.offsets + a.E);
        }
    }
    __syncthreads();
}

struct Item {
    int e;       // matrix
    int tile;    // tile of weight rows
    int row0;    // first row of the chunk
    int rows;    // its rows
};

// A CTA's items i = first, first + step, ... of `count`: experts in order,
// their weight tiles, then the chunks of rows that share such a tile (so that
// a tile's second reader finds it in the L2).  A whole warp steps through them;
// i is kept as chunk * w_tiles + rest, and the expert is found in two ballots
// (small K does not hide a search that reads one expert after the other).
struct Items {
    int i, count, step, w_tiles, chunk, rest, d_chunk, d_rest;

    __device__ __forceinline__ Items(int first, int step_, int count_, int w_tiles_)
        : i(first), count(count_), step(step_), w_tiles(w_tiles_), chunk(first / w_tiles_), rest(first % w_tiles_),
          d_chunk(step_ / w_tiles_), d_rest(step_ % w_tiles_) {}
    __device__ __forceinline__ bool more() const { return i < count; }
    __device__ __forceinline__ void next() {
        i += step;
        chunk += d_chunk;
        rest += d_rest;
        if (rest >= w_tiles) { rest -= w_tiles; ++chunk; }
    }
    __device__ __forceinline__ Item get(const Chunks* ch, int E) const {
        const int lane = threadIdx.x & 31;
        // the last expert with before[e] <= chunk: its group of 32, then itself
        const int g = __popc(__ballot_sync(0xffffffffu, 32 * lane < E && ch->before[min(32 * lane, E)] <= chunk)) - 1;
        const int at = 32 * g + lane;
        const int e = 32 * g + __popc(__ballot_sync(0xffffffffu, at < E && ch->before[min(at, E)] <= chunk)) - 1;
        Item it;
        it.e = e;
        it.row0 = ch->first[e];
        it.rows = ch->first[e + 1] - it.row0;
        it.tile = rest;
        const int before = ch->before[e], chunks = ch->before[e + 1] - before;
        if (chunks > 1) {   // chunks of near-equal size, fastest
            const int local = (chunk - before) * w_tiles + rest;
            it.tile = local / chunks;
            const bq::RowChunk part = bq::row_chunk(it.rows, chunks, local - it.tile * chunks);
            it.row0 += part.first;
            it.rows = part.rows;
        }
        return it;
    }
};

// ---------------------------------------------------------------- weights on the lanes
//
// Tile = 128 weight rows (MMA M, TMEM lanes) x up to 32 rows of x (MMA N, TMEM
// columns).  For few rows the time is that of reading the weights once: they
// go from HBM to shared memory by TMA and from there into the tensor cores,
// through no register, and the N side costs nothing where it is short.  With
// SwiGLU a tile holds 64 gate rows and their 64 up rows, 16 + 16 in each lane
// quarter, so that a gate value and its up value are 16 lanes apart.
//
// 224 threads, one CTA per SM, persistent over the items:
//   warp 0     TMA producer: 128 x 128 bytes of weights and the rows' 128
//              bytes into a ring of 10 stages (one stage = one block of K);
//   warp 1     owns the TMEM, issues the MMAs of a stage into the next of 8
//              accumulator slots;
//   warp 2     copies the slot's scales (xs of every row, ws) beside it;
//   warps 3-6  add slot by slot to their sums, then write y.
// With few items K is split over a cluster: the CTAs leave their sums in
// shared memory and each finishes a share of the rows, in rank order.
//
// Measured: up to 48 of 256 experts with a row or two each, 4096 x 2048: 62.2
// us, 6.0 TB/s.  One row x 4096 x 4096: 5.7 us, of which reading the weights
// would take 2.5.  An epilogue warp takes its blocks one after the other (wait,
// TMEM load, scales, sums, release), 0.22 us each, eight of them with K split
// over four CTAs; launch, first loads and the cluster's two barriers are the
// rest.  128 rows, unsplit, 32 blocks: 11.4 us.
constexpr int kLaneRows = 32;      // rows of x in a tile (the columns of a TMEM slot)
constexpr int kLaneThreads = 224;

struct LaneSmem {
    static constexpr int S = 10, A = 8, BOX = 16;                 // stages, TMEM slots, rows of a box
    static constexpr int kWBytes = kBlock * 128;
    static constexpr int kStage = kWBytes + kLaneRows * 128;
    static constexpr int kScaleSlot = kLaneRows + 4;              // xs of the rows, ws of gate and up
    static constexpr int kScales = S * kStage;
    static constexpr int kTiles = kScales + A * kScaleSlot * 4;
    static constexpr int kBars = kTiles + (int)sizeof(Chunks);
    static constexpr int kNumBars = 2 * S + 3 * A + 1;
    static constexpr int kBytes = 1024 + kBars + 8 * kNumBars + 16;
};
static_assert(LaneSmem::kBytes <= 232448 && LaneSmem::kTiles % 16 == 0, "smem");

// Bias of the weight row that a lane holds: column c of y, with SwiGLU its gate value (lanes 0-15) or its up value.
template <bool SWIGLU>
__device__ __forceinline__ float lane_bias(const EndArgs& a, int e, int c) {
    if (!a.bias || c >= a.cols) return 0.f;
    const int up = SWIGLU && (threadIdx.x & 16) ? a.cols : 0;
    return load_early(a.bias + (int64_t)e * a.n + up + c);
}

// EPI: with an end (bias, activation, scale, residual).
template <bool SWIGLU, bool EPI>
__global__ void __launch_bounds__(kLaneThreads, 1)
mm_lanes_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const ArgsOf<EPI> a,
                int split) {
    using M = LaneSmem;
    constexpr int S = M::S, A = M::A, NT = kLaneRows;
    constexpr uint32_t kCols = NT * A;
    static_assert(kCols == 256, "TMEM columns");
    extern __shared__ uint8_t smem_dyn[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
    float* scales = reinterpret_cast<float*>(smem + M::kScales);
    Chunks* chunks = reinterpret_cast<Chunks*>(smem + M::kTiles);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + M::kBars);
    const uint32_t bar0 = smem_u32(bars), ring = smem_u32(smem);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (S + s); };
    auto acc_full = [&](int q) { return bar0 + 8u * (2 * S + q); };
    auto acc_empty = [&](int q) { return bar0 + 8u * (2 * S + A + q); };
    auto sc_full = [&](int q) { return bar0 + 8u * (2 * S + 2 * A + q); };
    const uint32_t drain = bar0 + 8u * (2 * S + 3 * A);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + M::kNumBars);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    volatile uint32_t* filled = tmem_slot + 2;   // stages that the producer has filled

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) { mbar_init(full(i), 1); mbar_init(empty(i), 1); }
        for (int i = 0; i < A; ++i) { mbar_init(acc_full(i), 1); mbar_init(acc_empty(i), 4); mbar_init(sc_full(i), 32); }
        mbar_init(drain, 1);
        *abort_flag = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(tmem_slot)), "r"(kCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // launched behind whatever precedes it on the stream: nothing before this line touches global memory
    bq::grid_dependency_wait();
    bq::allow_dependents();
    count_chunks(a, 32, chunks);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    constexpr int kTileCols = SWIGLU ? 64 : 128;
    const int w_tiles = (a.cols + kTileCols - 1) / kTileCols;
    const int items = chunks->before[a.E] * w_tiles;   // the host made sure that it is an int
    const int rank = split > 1 ? (int)cluster_rank() : 0;
    const int first = blockIdx.x / split, step = gridDim.x / split;
    const int b0 = a.kb * rank / split, b1 = a.kb * (rank + 1) / split;
    const unsigned long long limit = a.wait_limit_ns;

    float bias = 0.f;   // of the column that an epilogue thread has (an end's)
    auto ended = [&](float v, float residual) {
        if constexpr (EPI) v = __fmaf_rn(a.scale, v, residual);
        return v;
    };
    const bool one = elect_one();
    bool ok = !(a.skip_copies == 3 && split > 1 ? rank & 1 : a.skip_copies);
    if (warp == 0) {
        int s = 0, issued = 0;
        uint32_t ph = 1;   // a fresh barrier passes for the phase before its first
        for (Items i(first, step, items, w_tiles); ok && i.more(); i.next()) {
            const Item it = i.get(chunks, a.E);
            const int boxes = (it.rows + M::BOX - 1) / M::BOX;
            const uint32_t bytes = M::kWBytes + boxes * M::BOX * 128;
            for (int b = b0; b < b1; ++b) {
                if (!(ok = warp_wait_all(empty(s), ph, abort_flag, a.status, limit))) break;
                if (one) {
                    const uint32_t dst = ring + s * M::kStage;
                    mbar_expect_tx(full(s), bytes);
                    if (SWIGLU) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            tma_load_4d(dst + q * 4096, &map_w, b * kBlock, 64 * it.tile + 16 * q, 0, it.e, full(s));
                    } else {
                        tma_load_3d(dst, &map_w, b * kBlock, 128 * it.tile, it.e, full(s));
                    }
                    for (int q = 0; q < boxes; ++q)
                        tma_load_2d(dst + M::kWBytes + q * M::BOX * 128, &map_x, b * kBlock, it.row0 + q * M::BOX, full(s));
                }
                ++issued;
                if (++s == S) { s = 0; ph ^= 1u; }
            }
        }
        if (one) *filled = issued;
    } else if (warp == 1) {
        const uint64_t wd0 = smem_desc_sw128(ring), xd0 = smem_desc_sw128(ring + M::kWBytes);
        int s = 0, q = 0;
        uint32_t ph = 0, aph = 1;
        ok = true;
        for (Items i(first, step, items, w_tiles); ok && i.more(); i.next()) {
            const Item it = i.get(chunks, a.E);
            const uint32_t idesc = idesc_e4m3((it.rows + 15) & ~15);
            for (int b = b0; b < b1; ++b) {
                if (!(ok = warp_wait_both(full(s), ph, acc_empty(q), aph, abort_flag, a.status, limit))) break;
                tc_fence_after();
                if (one) {
                    const uint32_t stage = s * (M::kStage >> 4);
#pragma unroll
                    for (int j = 0; j < 4; ++j)     // +32 bytes along K
                        mma_e4m3(tmem + q * NT, wd0 + stage + 2 * j, xd0 + stage + 2 * j, idesc, j != 0);
                    mma_commit(acc_full(q));
                    mma_commit(empty(s));
                }
                __syncwarp();
                if (++s == S) { s = 0; ph ^= 1u; }
                if (++q == A) { q = 0; aph ^= 1u; }
            }
        }
    } else if (warp == 2) {
        int q = 0;
        uint32_t aph = 1;
        ok = true;
        for (Items i(first, step, items, w_tiles); ok && i.more(); i.next()) {
            const Item it = i.get(chunks, a.E);
            const float* xs = a.xs + (int64_t)it.row0 * a.kb;
            // weight rows 128 tile.. are scale row `tile`; of a gate/up weight, gate rows 64 tile.. are scale row
            // tile / 2 and their up rows n/2 further on
            const int wrow = lane == 0 ? (SWIGLU ? it.tile / 2 : it.tile) : it.tile / 2 + a.nb / 2;
            const float* ws = a.ws + ((int64_t)it.e * a.nb + wrow) * a.kb;
            for (int b = b0; b < b1; ++b) {
                if (!(ok = warp_wait_all(acc_empty(q), aph, abort_flag, a.status, limit))) break;
                const uint32_t dst = smem_u32(scales + q * M::kScaleSlot);
                if (lane < it.rows) copy4_async(dst + 4 * lane, xs + lane * a.kb + b);
                if (lane < (SWIGLU ? 2 : 1)) copy4_async(dst + 4 * (NT + lane), ws + b);
                copies_arrive(sc_full(q));
                if (++q == A) { q = 0; aph ^= 1u; }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        const int quarter = warp & 3, p = 32 * quarter + lane;
        const uint32_t base = tmem + ((uint32_t)(32 * quarter) << 16);
        int q = 0;
        uint32_t aph = 0;
        ok = true;
        for (Items i(first, step, items, w_tiles); ok && i.more(); i.next()) {
            const Item it = i.get(chunks, a.E);
            const int c = SWIGLU ? 64 * it.tile + 16 * quarter + (lane & 15) : 128 * it.tile + p;
            if constexpr (EPI) {   // on their way while the weights are
                bias = lane_bias<SWIGLU>(a, it.e, c);
                const int c0 = SWIGLU ? c - (lane & 15) : c - lane;
                if (a.residual && lane < it.rows && c0 < a.cols)
                    prefetch_residual(a, (int64_t)it.row0 + lane, c0, SWIGLU ? 16 : 32);
            }
            float acc[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] = 0.f;
            for (int b = b0; b < b1; ++b) {
                if (!(ok = warp_wait_both(sc_full(q), aph, acc_full(q), aph, abort_flag, a.status, limit))) break;
                tc_fence_after();
                const float* sc = scales + q * M::kScaleSlot;
                uint32_t v[32];
                tmem_ld32(base + q * NT, v);
                const float ws = sc[NT + (SWIGLU ? (lane >> 4) : 0)];
                float x[NT];
#pragma unroll
                for (int j = 0; j < NT; j += 4) {
                    const float4 x4 = *reinterpret_cast<const float4*>(sc + j);
                    x[j] = x4.x * ws; x[j + 1] = x4.y * ws; x[j + 2] = x4.z * ws; x[j + 3] = x4.w * ws;
                }
                tmem_wait_ld(v);
#pragma unroll
                for (int j = 0; j < NT; ++j) acc[j] = __fmaf_rn(__uint_as_float(v[j]), x[j], acc[j]);
                tc_fence_before();
                __syncwarp();
                if (one) mbar_arrive(acc_empty(q));
                if (++q == A) { q = 0; aph ^= 1u; }
            }
            if (!ok) break;
            if (split > 1) {   // sums to shared memory (every copy and MMA of this CTA has ended): [row][lane]
                float* red = reinterpret_cast<float*>(smem);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (t < it.rows) red[t * 128 + p] = acc[t];
                break;         // one item per cluster
            }
            float res[NT];
            if constexpr (EPI) {
#pragma unroll
                for (int t = 0; t < NT; ++t) acc[t] += bias;
                // of the values that this thread stores: with SwiGLU those of every other row
                if (SWIGLU) {
                    float every[NT / 2];
                    load_residual(a, (int64_t)it.row0 + (lane >> 4), 2, (int64_t)it.row0 + it.rows, c, every);
#pragma unroll
                    for (int t = 0; t < NT; ++t) res[t] = every[t / 2];
                } else {
                    load_residual(a, (int64_t)it.row0, 1, (int64_t)it.row0 + it.rows, c, res);
                }
                if (!SWIGLU) activate<END_ANY>(acc, a.act);
            }
            if (SWIGLU) {
                // lanes 0-15 hold gate rows, 16-31 their up rows; each half finishes every other row of x
#pragma unroll
                for (int t = 0; t < NT; t += 2) {
                    if (t < it.rows) {
                        const float recv = __shfl_xor_sync(0xffffffffu, lane < 16 ? acc[t + 1] : acc[t], 16);
                        const float g = lane < 16 ? acc[t] : recv, u = lane < 16 ? recv : acc[t + 1];
                        const int r = t + (lane >> 4);
                        const float v = ended((EPI ? silu_end(g) : silu_f(g)) * u, res[t]);
                        if (r < it.rows) bq::store_value(a.y, (int64_t)(it.row0 + r) * a.ldy + c, a.ydtype, v);
                    }
                }
            } else if (c < a.cols) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (t < it.rows)
                        bq::store_value(a.y, (int64_t)(it.row0 + t) * a.ldy + c, a.ydtype, ended(acc[t], res[t]));
            }
        }
    }

    if (split > 1) {
        __syncwarp();
        cluster_sync();
        if (warp >= 3 && first < items) {
            // a CTA whose waits ran out left no sums: then y is not written, as without a split (asked for beside the
            // first sums, which take as long to come)
            const uint32_t aborted = lane < split ? peer_load_u32(smem_u32(tmem_slot + 1), lane) : 0u;
            const int quarter = warp & 3, p = 32 * quarter + lane;
            const Item it = Items(first, step, items, w_tiles).get(chunks, a.E);
            const int c = SWIGLU ? 64 * it.tile + 16 * quarter + (lane & 15) : 128 * it.tile + p;
            constexpr int kAtOnce = 4;   // rows whose loads are in flight together
            for (int t0 = rank; t0 < it.rows; t0 += kAtOnce * split) {
                float part[kAtOnce][kMaxCluster] = {};
                float res[kAtOnce];
                if constexpr (EPI) load_residual(a, (int64_t)it.row0 + t0, split, (int64_t)it.row0 + it.rows, c, res);
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j) {
                    const uint32_t at = ring + 4 * ((t0 + j * split) * 128 + p);
                    if (t0 + j * split >= it.rows) break;
#pragma unroll
                    for (int r = 0; r < kMaxCluster; ++r) {
                        if (r >= split) break;
                        part[j][r] = peer_load(at, r);
                    }
                }
                if (__any_sync(0xffffffffu, aborted != 0)) break;
                float v[kAtOnce];
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j) {
                    v[j] = part[j][0];
#pragma unroll
                    for (int r = 1; r < kMaxCluster; ++r) v[j] += part[j][r];
                    if (EPI) v[j] += bias;
                    if (SWIGLU) {
                        const float u = __shfl_xor_sync(0xffffffffu, v[j], 16);
                        v[j] = (EPI ? silu_end(v[j]) : silu_f(v[j])) * u;
                    }
                }
                if constexpr (EPI && !SWIGLU) activate<END_ANY>(v, a.act);
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j) {
                    const int t = t0 + j * split;
                    if (t >= it.rows) break;
                    v[j] = ended(v[j], res[j]);
                    if (c < a.cols && (!SWIGLU || lane < 16))
                        bq::store_value(a.y, (int64_t)(it.row0 + t) * a.ldy + c, a.ydtype, v[j]);
                }
            }
        }
        __syncwarp();
        cluster_sync();   // peers may still be reading this CTA's sums
    }
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {   // a warp gave up: what the others started ends before the memory it uses is freed (bounded)
        volatile uint32_t no_abort = 0;
        if (warp == 0) {
            const int issued = *filled;
            for (int u = max(0, issued - S); u < issued; ++u)
                mbar_wait(full(u % S), (u / S) & 1, &no_abort, a.status, limit);
        } else if (warp == 1 && elect_one()) {
            mma_commit(drain);
            mbar_wait(drain, 0, &no_abort, a.status, limit);
        }
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols) : "memory");
    }
}

// ---------------------------------------------------------------- rows on the lanes
//
// For many rows the tensor cores bound it.  With the rows of x on the lanes a
// block's scale is one number per thread and scale block, so adding a block
// costs one multiply-add per value and nothing else (against a scale fetched
// per column above).  Tile = up to 128 rows of x (MMA M, TMEM lanes) x 256
// weight rows (TMEM columns).
//
// A slot of TMEM is busy from its MMAs through the commit, the epilogue's
// loads and the word back to the issuer.  There is room for two slots of 256
// columns, so the tile's two halves of 128 columns (MMA N) are pipelines of
// their own, with an issuing warp, two slots and four epilogue warps each: one
// half's MMAs run while the other's slots change hands.  With SwiGLU each half
// is 64 gate rows and their 64 up rows, and a thread holds both.
//
// 384 threads, one CTA per SM, persistent over the items:
//   warp 0      TMA producer: 128 bytes of 128 rows and of 256 weight rows into
//               a ring of 4 stages (48 KB each);
//   warps 1-2   issue the MMAs of a half; warp 1 owns the TMEM;
//   warp 3      idle (warpgroups give and take registers as a whole);
//   warps 4-11  one thread per row and half: 128 fp32 sums in registers, then
//               y.  They take the registers that the first warpgroup gives up:
//               with fewer the sums spill, which made a block 2.4 times as
//               long.
// In the long run a block of 128 x 256 x 128 takes 0.36 us of an SM, 0.91 of
// twice the measured bf16 rate, and the MMAs bound it: without the multiply-
// adds it takes as long, with a quarter of the MMAs 0.32 us.  On top come the
// rounds of tiles (2048 x 4096 x 4096: 256 on 152 SMs), about 6 us of launch,
// first loads and last stores for the first round, and about 2 us for each
// further one, while a tile is stored and the next one's scales are fetched and
// the MMAs run only two blocks ahead.  2048 x 4096 x 4096: 31.5 us (2.2
// PFLOP/s; 8192 rows 2.6).  A tile is 256 columns wide whatever the rows, so
// 256 to 1024 rows take 15.3 to 17.6 us.
constexpr int kWideThreads = 384;
constexpr int kWideRegs = 224, kControlRegs = 56;   // 256 * 224 + 128 * 56 = 384 * 168, what the launch holds
static_assert(256 * kWideRegs + 128 * kControlRegs <= kWideThreads * 168, "registers");

constexpr int kOutRow = 144;   // 128 bytes of a row of y, padded: eight rows' 16 bytes lie in distinct banks

struct WideSmem {
    static constexpr int S = 4, A = 2;                              // stages; slots of a half
    static constexpr int kXBytes = 128 * 128;
    static constexpr int kHalfBytes = 128 * 128;                    // weight rows of a half
    static constexpr int kStage = kXBytes + 2 * kHalfBytes;
    static constexpr int kTiles = S * kStage;
    static constexpr int kOut = kTiles + (int)sizeof(Chunks);       // the epilogue warps' pieces of y
    static constexpr int kBars = kOut + 8 * 16 * kOutRow;           // 16-byte aligned: the slots' barriers differ in bit 3
    static constexpr int kNumBars = 2 * S + 4 * A + 2;
    static constexpr int kBytes = 1024 + kBars + 8 * kNumBars + 16;
};
static_assert(WideSmem::kBytes <= 232448 && WideSmem::kBars % 16 == 0 && WideSmem::S % 2 == 0, "smem");

__device__ __forceinline__ void add_scaled(float* acc, const uint32_t (&v)[32], float f) {
#pragma unroll
    for (int i = 0; i < 32; ++i) acc[i] = __fmaf_rn(__uint_as_float(v[i]), f, acc[i]);
}

__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Two ways to y for a warp's 32 rows, a row per lane:
//   16-bit rows on 32-byte boundaries: each lane stores its row, 32 bytes at a
//   time (whole sectors);
//   other rows, and fp32: by way of shared memory, below, so that eight lanes
//   store 128 contiguous bytes.
// Both ways in one run each, 2048 x 4096 x 4096: fp32 34.3 us by way of shared
// memory and 37.1 direct; 4095 columns of 16 bits, on no boundary, 60.4 and 104;
// bf16 31.3 and 31.6, and the gate/up product of 128 experts, whose epilogue has
// less time, 90.3 and 87.0.
//
// 128 bytes of each row (w) to rows row0.. of y from column c on, those below `rows`, 16 rows at a time.
__device__ __forceinline__ void store_rows(const Args& a, uint8_t* buf, const uint4 (&w)[8], int64_t row0, int rows, int c,
                                           bool aligned) {
    const int lane = threadIdx.x & 31, es = a.ydtype == BQ_DT_F32 ? 4 : 2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (lane >> 4 == h) {
            uint4* to = reinterpret_cast<uint4*>(buf + (lane & 15) * kOutRow);
#pragma unroll
            for (int j = 0; j < 8; ++j) to[j] = w[j];
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * i + (lane >> 3), col = c + (lane & 7) * (16 / es);
            const uint4 v = *reinterpret_cast<const uint4*>(buf + r * kOutRow + (lane & 7) * 16);
            if (16 * h + r >= rows || col >= a.cols) continue;
            uint8_t* to = static_cast<uint8_t*>(a.y) + ((row0 + 16 * h + r) * a.ldy + col) * es;
            if (aligned && col + 16 / es <= a.cols) {
                *reinterpret_cast<uint4*>(to) = v;
            } else {
                const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (es == 4) {
                        if (col + e < a.cols) reinterpret_cast<uint32_t*>(to)[e] = x[e];
                    } else {
                        if (col + 2 * e < a.cols) reinterpret_cast<uint16_t*>(to)[2 * e] = (uint16_t)x[e];
                        if (col + 2 * e + 1 < a.cols) reinterpret_cast<uint16_t*>(to)[2 * e + 1] = (uint16_t)(x[e] >> 16);
                    }
                }
            }
        }
        __syncwarp();
    }
}

__device__ __forceinline__ void load32(const void* p, uint4& lo, uint4& hi) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(lo.x), "=r"(lo.y), "=r"(lo.z), "=r"(lo.w), "=r"(hi.x), "=r"(hi.y), "=r"(hi.z), "=r"(hi.w)
                 : "l"(p) : "memory");
}

// 128 bytes of a row of the residual from column c on (32 fp32 values, or 64), added to v: those columns that exist.
// vectors: the matrix allows 32-byte loads (whole sectors), which then are in flight together.  (fp32 rows by way of
// shared memory, eight lanes 128 bytes, took longer: 49 us against 44 for 2048 x 4096 x 4096.)
template <int N>
__device__ __forceinline__ void add_residual(const EndArgs& a, int64_t row, int c, bool vectors, float* v) {
    const int64_t at = row * a.ldr + c;
    if (vectors && c + N <= a.cols) {
        const uint8_t* p = static_cast<const uint8_t*>(a.residual) + at * (128 / N);
        constexpr int kPer = N / 8;
        uint4 raw[8];
#pragma unroll
        for (int i = 0; i < 8; i += 2) load32(p + 16 * i, raw[i], raw[i + 1]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float f[kPer];
            if constexpr (N == 32) bq::RowVec<BQ_DT_F32>::unpack(raw[i], f);
            else if (a.ydtype == BQ_DT_F16) bq::RowVec<BQ_DT_F16>::unpack(raw[i], f);
            else bq::RowVec<BQ_DT_BF16>::unpack(raw[i], f);
#pragma unroll
            for (int j = 0; j < kPer; ++j) v[kPer * i + j] = __fmaf_rn(a.scale, v[kPer * i + j], f[j]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (c + i < a.cols) v[i] = __fmaf_rn(a.scale, v[i], load_value(a.residual, at + i, a.ydtype));
}

// Bias of the values that a thread sums: acc[j] is column c0 + j of y, with SwiGLU the gate value of column c0 + j % 64
// or its up value.  Each warp fetches its own copy to where its rows go through later: copies that nothing waits for
// until the sums are done, and that need no registers meanwhile (a load into registers at this place made a block of K
// 8% longer).  end_rows waits for them: one call of each per item.
template <bool SWIGLU>
__device__ __forceinline__ void fetch_bias(const EndArgs& a, int e, int c0, uint8_t* buf) {
    if (!a.bias) return;
    const float* bias = a.bias + (int64_t)e * a.n;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = 32 * i + (threadIdx.x & 31), c = min(c0 + (SWIGLU ? j & 63 : j), a.cols - 1);
        copy4_async(smem_u32(buf) + 4 * j, bias + (SWIGLU && i >= 2 ? a.cols : 0) + c);
    }
}

// A row's end, in place: column c0 + n of y in acc[n].
template <bool SWIGLU, int END, bool RESIDUAL>
__device__ __forceinline__ void end_rows(const EndArgs& a, float (&acc)[128], const uint8_t* buf, int64_t row, bool live, int c0,
                                         bool vectors) {
    constexpr int kCols = SWIGLU ? 64 : 128;
    if (a.bias) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        const float4* b4 = reinterpret_cast<const float4*>(buf);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const float4 b = b4[j];
            acc[4 * j] += b.x;
            acc[4 * j + 1] += b.y;
            acc[4 * j + 2] += b.z;
            acc[4 * j + 3] += b.w;
        }
        __syncwarp();   // the rows go through buf next
    }
    if (SWIGLU) {
#pragma unroll
        for (int n = 0; n < 64; ++n) acc[n] = silu_end(acc[n]) * acc[64 + n];
    } else {
        activate<END>(acc, a.act);
    }
    if (!RESIDUAL) {
        if (a.scale != 1.f) {
#pragma unroll
            for (int n = 0; n < kCols; ++n) acc[n] *= a.scale;
        }
    } else if (live && a.ydtype == BQ_DT_F32) {
#pragma unroll
        for (int n = 0; n < kCols; n += 32) add_residual<32>(a, row, c0 + n, vectors, acc + n);
    } else if (live) {
#pragma unroll
        for (int n = 0; n < kCols; n += 64) add_residual<64>(a, row, c0 + n, vectors, acc + n);
    }
}

// END, RESIDUAL: the end (bias, activation, scale, residual) that it is compiled for.
template <bool SWIGLU, int END, bool RESIDUAL>
__global__ void __launch_bounds__(kWideThreads, 1)
mm_wide_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
               const ArgsOf<(END > 0)> a) {
    using M = WideSmem;
    constexpr int S = M::S, A = M::A, kTileCols = SWIGLU ? 128 : 256;
    extern __shared__ uint8_t smem_dyn[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
    Chunks* chunks = reinterpret_cast<Chunks*>(smem + M::kTiles);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + M::kBars);
    const uint32_t bar0 = smem_u32(bars), ring = smem_u32(smem);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (S + s); };
    auto acc_full = [&](int half, int q) { return bar0 + 8u * (2 * S + A * half + q); };
    auto acc_empty = [&](int half, int q) { return bar0 + 8u * (2 * S + A * (2 + half) + q); };
    auto drain = [&](int half) { return bar0 + 8u * (2 * S + 4 * A + half); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + M::kNumBars);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    volatile uint32_t* filled = tmem_slot + 2;   // stages that the producer has filled

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) { mbar_init(full(i), 1); mbar_init(empty(i), 2); }
        for (int i = 0; i < 2 * A; ++i) { mbar_init(acc_full(0, i), 1); mbar_init(acc_empty(0, i), 4); }
        mbar_init(drain(0), 1);
        mbar_init(drain(1), 1);
        *abort_flag = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(tmem_slot)), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // launched behind whatever precedes it on the stream: nothing before this line touches global memory
    bq::grid_dependency_wait();
    bq::allow_dependents();
    count_chunks(a, 128, chunks);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int w_tiles = (a.cols + kTileCols - 1) / kTileCols;
    const int items = chunks->before[a.E] * w_tiles;   // the host made sure that it is an int
    const int first = blockIdx.x, step = gridDim.x;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs));
        const bool one = elect_one();
        bool ok = !a.skip_copies;
        if (warp == 0) {
            int s = 0, issued = 0;
            uint32_t ph = 1;   // a fresh barrier passes for the phase before its first
            for (Items i(first, step, items, w_tiles); ok && i.more(); i.next()) {
                const Item it = i.get(chunks, a.E);
                const int w_row = kTileCols * it.tile;
                for (int b = 0; b < a.kb; ++b) {
                    if (!(ok = warp_wait_all(empty(s), ph, abort_flag, a.status, a.wait_limit_ns))) break;
                    if (one) {
                        const uint32_t dst = ring + s * M::kStage;
                        mbar_expect_tx(full(s), M::kStage);
                        tma_load_2d(dst, &map_x, b * kBlock, it.row0, full(s));
                        for (int h = 0; h < 2; ++h) {
                            if (SWIGLU)   // 64 gate rows and their 64 up rows
                                tma_load_4d(dst + M::kXBytes + h * M::kHalfBytes, &map_w, b * kBlock, w_row + 64 * h, 0, it.e,
                                            full(s));
                            else
                                tma_load_3d(dst + M::kXBytes + h * M::kHalfBytes, &map_w, b * kBlock, w_row + 128 * h, it.e,
                                            full(s));
                        }
                    }
                    ++issued;
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
            }
            if (one) *filled = issued;
        } else if (warp < 3) {
            // Lean: what one warp does per block, in order, bounds the MMA rate.
            const int half = warp - 1;
            const uint32_t idesc = idesc_e4m3(128);
            const uint64_t xd0 = smem_desc_sw128(ring);
            const uint64_t wd0 = smem_desc_sw128(ring + M::kXBytes + half * M::kHalfBytes);
            int s = 0;
            uint32_t ph = 0, aph = 1;   // phases of the stages, and of the slots (a fresh barrier passes)
            uint32_t stage_full = full(0), stage_empty = empty(0), slot_full = acc_full(half, 0), slot_empty = acc_empty(half, 0);
            uint32_t d = tmem + half * A * 128, stage = 0;   // stage: in units of a descriptor's address
            ok = true;
            const int64_t total = first < items ? (int64_t)((items - first + step - 1) / step) * a.kb : 0;
#pragma unroll 1
            for (int64_t j = 0; j < total; ++j) {   // the blocks of all items alike
                if (!(ok = warp_wait_both(stage_full, ph, slot_empty, aph, abort_flag, a.status, a.wait_limit_ns))) break;
                tc_fence_after();
                if (one) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)   // +32 bytes along K
                        mma_e4m3(d, xd0 + stage + 2 * i, wd0 + stage + 2 * i, idesc, i != 0);
                    mma_commit(slot_full);
                    mma_commit(stage_empty);
                }
                __syncwarp();
                aph ^= (slot_full >> 3) & 1u;   // after the second slot (the first one's barrier has bit 3 clear)
                slot_full ^= 8u;
                slot_empty ^= 8u;
                d ^= 128u;
                stage += M::kStage >> 4;
                stage_full += 8u;
                stage_empty += 8u;
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                    stage = 0;
                    stage_full = full(0);
                    stage_empty = empty(0);
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWideRegs));
        const int quarter = warp & 3, half = (warp - 4) >> 2, p = 32 * quarter + lane;
        const int es = a.ydtype == BQ_DT_F32 ? 4 : 2;
        const uintptr_t y_align = reinterpret_cast<uintptr_t>(a.y) | (uintptr_t)(a.ldy * es);
        const bool aligned = y_align % 16 == 0, sectors = y_align % 32 == 0;
        bool vectors = false;
        if constexpr (RESIDUAL) vectors = (reinterpret_cast<uintptr_t>(a.residual) | (uintptr_t)(a.ldr * es)) % 32 == 0;
        // The slot in turn: its barriers (the second's 8 bytes behind the first's) and its columns, flipped by a bit.
        uint32_t bar_full = acc_full(half, 0), t = tmem + ((uint32_t)(32 * quarter) << 16) + half * A * 128, aph = 0;
        uint32_t bar_free = acc_empty(half, 0);
        const bool one = elect_one();
        bool ok = true;
        for (Items i(first, step, items, w_tiles); ok && i.more(); i.next()) {
            const Item it = i.get(chunks, a.E);
            const float* xs = a.xs + (int64_t)(it.row0 + min(p, it.rows - 1)) * a.kb;
            const float* ws = a.ws + (int64_t)it.e * a.nb * a.kb;
            // this half's first column and the scale row of its columns, with SwiGLU of its gate columns and up columns
            const int c0 = kTileCols * it.tile + kTileCols / 2 * half;
            const int o_lo = min(c0 / kBlock, a.nb - 1) * a.kb, o_hi = o_lo + a.nb / 2 * a.kb;
            uint8_t* buf = smem + M::kOut + (warp - 4) * 16 * kOutRow;
            // On their way while the blocks are.  A warp without rows of this item has no use for a bias, and does not
            // come to the wait in end_rows: copies left in flight would meet those of its next item in the same place.
            if constexpr (END != END_NONE) {
                if (32 * quarter < it.rows) {
                    fetch_bias<SWIGLU>(a, it.e, c0, buf);
                    if (RESIDUAL && p < it.rows) prefetch_residual(a, (int64_t)it.row0 + p, c0, SWIGLU ? 64 : 128);
                }
            }
            float acc[128];
#pragma unroll
            for (int j = 0; j < 128; ++j) acc[j] = 0.f;
            // Scales are loaded two blocks ahead; a block's wait and the load of its first columns come before the last
            // sums of the block before it, which cover their latency.
            const int b_last = a.kb - 1, b_next = min(1, b_last);
            float x0 = __ldg(xs), lo0 = __ldg(ws + o_lo), hi0 = SWIGLU ? __ldg(ws + o_hi) : 0.f;
            float x1 = load_early(xs + b_next), lo1 = load_early(ws + o_lo + b_next), hi1 = 0.f;
            if (SWIGLU) hi1 = load_early(ws + o_hi + b_next);
            uint32_t v0[32], v1[32];
            if (!(ok = warp_wait_all(bar_full, aph, abort_flag, a.status, a.wait_limit_ns))) break;
            tc_fence_after();
            tmem_ld32(t, v0);
#pragma unroll 1
            for (int b = 0; b < a.kb; ++b) {
                const float f_lo = x0 * lo0, f_hi = SWIGLU ? x0 * hi0 : f_lo;
                x0 = x1; lo0 = lo1; hi0 = hi1;
                const int bn = min(b + 2, b_last);
                x1 = load_early(xs + bn);
                lo1 = load_early(ws + o_lo + bn);
                if (SWIGLU) hi1 = load_early(ws + o_hi + bn);
                tmem_wait_ld(v0);
                tmem_ld32(t + 32, v1);
                add_scaled(acc, v0, f_lo);
                tmem_wait_ld(v1);
                tmem_ld32(t + 64, v0);
                add_scaled(acc + 32, v1, f_lo);
                tmem_wait_ld(v0);
                tmem_ld32(t + 96, v1);
                add_scaled(acc + 64, v0, f_hi);
                tmem_wait_ld(v1);
                tc_fence_before();
                __syncwarp();
                if (one) mbar_arrive(bar_free);
                aph ^= (bar_full >> 3) & 1u;   // after the second slot (the first one's barrier has bit 3 clear)
                bar_full ^= 8u;
                bar_free ^= 8u;
                t ^= 128u;
                if (b < b_last) {
                    if (!(ok = warp_wait_all(bar_full, aph, abort_flag, a.status, a.wait_limit_ns))) break;
                    tc_fence_after();
                    tmem_ld32(t, v0);
                }
                add_scaled(acc + 96, v1, f_hi);
            }
            if (!ok) break;
            const int rows = it.rows - 32 * quarter;   // of this warp
            if (rows > 0) {
                const int64_t row0 = it.row0 + 32 * quarter;
                if constexpr (END != END_NONE) end_rows<SWIGLU, END, RESIDUAL>(a, acc, buf, row0 + lane, lane < rows, c0, vectors);
                auto out = [&](int n) { return SWIGLU && END == END_NONE ? silu_f(acc[n]) * acc[(64 + n) & 127] : acc[n]; };
                auto out8 = [&](int n) {
                    const float f[8] = {out(n), out(n + 1), out(n + 2), out(n + 3), out(n + 4), out(n + 5), out(n + 6), out(n + 7)};
                    return a.ydtype == BQ_DT_F16 ? bq::RowVec<BQ_DT_F16>::pack(f) : bq::RowVec<BQ_DT_BF16>::pack(f);
                };
                constexpr int kOutCols = SWIGLU ? 64 : 128;
                if (a.ydtype == BQ_DT_F32) {
#pragma unroll
                    for (int n = 0; n < kOutCols; n += 32) {
                        uint4 w[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            w[j] = make_uint4(__float_as_uint(out(n + 4 * j)), __float_as_uint(out(n + 4 * j + 1)),
                                              __float_as_uint(out(n + 4 * j + 2)), __float_as_uint(out(n + 4 * j + 3)));
                        store_rows(a, buf, w, row0, rows, c0 + n, aligned);
                    }
                } else if (sectors && c0 + kOutCols <= a.cols) {
                    if (lane < rows) {
                        uint8_t* to = static_cast<uint8_t*>(a.y) + ((row0 + lane) * a.ldy + c0) * 2;
#pragma unroll
                        for (int n = 0; n < kOutCols; n += 16) {
                            const uint4 l = out8(n), h = out8(n + 8);
                            const uint32_t w[8] = {l.x, l.y, l.z, l.w, h.x, h.y, h.z, h.w};
                            store32(to + 2 * n, w);
                        }
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < kOutCols; n += 64) {
                        uint4 w[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) w[j] = out8(n + 8 * j);
                        store_rows(a, buf, w, row0, rows, c0 + n, aligned);
                    }
                }
            }
        }
        if (END != END_NONE) asm volatile("cp.async.wait_all;" ::: "memory");   // a wait that ran out leaves a bias on its way
    }
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {   // a warp gave up: what the others started ends before the memory it uses is freed (bounded)
        volatile uint32_t no_abort = 0;
        if (warp == 0) {
            const int issued = *filled;
            for (int u = max(0, issued - S); u < issued; ++u)
                mbar_wait(full(u % S), (u / S) & 1, &no_abort, a.status, a.wait_limit_ns);
        } else if (warp < 3 && elect_one()) {
            mma_commit(drain(warp - 1));
            mbar_wait(drain(warp - 1), 0, &no_abort, a.status, a.wait_limit_ns);
        }
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
}

// ---------------------------------------------------------------- launches of the wide kernel
constexpr int kSms = 152;

template <bool SWIGLU, int END, bool RESIDUAL>
cudaError_t launch_wide(const CUtensorMap& map_w, const CUtensorMap& map_x, const EndArgs& a, int64_t items,
                        cudaStream_t st) {
    static std::atomic<bool> attr_set[64];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_set[dev].load(std::memory_order_acquire)) {
        const cudaError_t e =
            cudaFuncSetAttribute(mm_wide_kernel<SWIGLU, END, RESIDUAL>, cudaFuncAttributeMaxDynamicSharedMemorySize, WideSmem::kBytes);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(true, std::memory_order_release);
    }
    return bq::launch_after(mm_wide_kernel<SWIGLU, END, RESIDUAL>, dim3((unsigned)std::min<int64_t>(items, kSms)), dim3(kWideThreads),
                            WideSmem::kBytes, st, map_w, map_x, static_cast<const ArgsOf<(END > 0)>&>(a));
}

// Of products with an end, each in a file of its own (a kernel of 128 sums a thread takes 10 s to compile): no activation
// or one of no cost, and SwiGLU; and the others.
cudaError_t launch_wide_simple_end(const CUtensorMap& map_w, const CUtensorMap& map_x, const EndArgs& a, int64_t items,
                                   bool swiglu, cudaStream_t st);
cudaError_t launch_wide_activation_end(const CUtensorMap& map_w, const CUtensorMap& map_x, const EndArgs& a, int64_t items,
                                       cudaStream_t st);

}  // namespace fp8mm
}  // namespace bq
