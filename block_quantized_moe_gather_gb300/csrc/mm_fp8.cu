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
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "gemm_internal.cuh"
#include "row_types.cuh"
#include "tc_ptx.cuh"

namespace {

using namespace bq::tc;

constexpr int kBlock = 128;        // K per scale, per TMA box (one 128-byte swizzle row) and per TMEM stage
constexpr int kMaxExperts = 1024;
constexpr int kMaxCluster = 8;

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
    int skip_copies;          // test only: the producer issues no copies (waits run out)
    int max_chunks;           // row chunks that offsets in order can make (more: overlapping, so descending, ones)
};

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
                 : "=f"(v) : "r"(addr), "r"(rank) : "memory");
    return v;
}

__device__ __forceinline__ float silu_f(float g) { return __fdividef(g, 1.f + expf(-g)); }

// ---------------------------------------------------------------- work items
// The row chunks of every expert: s_tiles[e] = chunks of the experts before e,
// s_tiles[E] their total.  A chunk is at most `most` rows; an expert's rows are
// cut into chunks of near-equal size.
__device__ __forceinline__ int chunks_of(const Args& a, int e, int most) {
    const int lo = __ldg(a.offsets + e), hi = __ldg(a.offsets + e + 1);
    if (!(0 <= lo && lo <= hi && hi <= a.rows)) {
        bq::set_device_error(a.status, BQ_DEV_BAD_ROW);
        return 0;
    }
    return (hi - lo + most - 1) / most;
}

// Fills s_tiles (all threads of the CTA; ends with a barrier).
__device__ __forceinline__ void count_chunks(const Args& a, int most, int32_t* s_tiles) {
    if (!a.offsets) {
        if (threadIdx.x == 0) {
            s_tiles[0] = 0;
            s_tiles[1] = (a.rows + most - 1) / most;
        }
    } else if (threadIdx.x < 32) {
        // one warp: 32 experts at a time, all loads of a group of four issued together
        int total = 0;
        for (int e0 = 0; e0 < a.E; e0 += 128) {
            int c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = e0 + 32 * i + (int)threadIdx.x;
                c[i] = e < a.E ? chunks_of(a, e, most) : 0;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = e0 + 32 * i + (int)threadIdx.x;
                int incl = c[i];
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, incl, off);
                    if ((int)threadIdx.x >= off) incl += v;
                }
                if (e < a.E) s_tiles[e] = total + incl - c[i];
                total += __shfl_sync(0xffffffffu, incl, 31);
            }
        }
        if (threadIdx.x == 0) s_tiles[a.E] = total;
    }
    __syncthreads();
}

struct Item {
    int e;       // matrix
    int tile;    // tile of weight rows
    int row0;    // first row of the chunk
    int rows;    // its rows
};

// Item i: experts in order, their weight tiles, then the chunks of rows that
// share such a tile (so that a tile's second reader finds it in the L2).
__device__ __forceinline__ Item find_item(const Args& a, const int32_t* s_tiles, int w_tiles, int i) {
    Item it;
    int lo = 0, hi = a.E - 1;   // the last expert with s_tiles[e] * w_tiles <= i
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((int64_t)s_tiles[mid] * w_tiles <= i) lo = mid; else hi = mid - 1;
    }
    it.e = lo;
    const int chunks = s_tiles[lo + 1] - s_tiles[lo], local = i - s_tiles[lo] * w_tiles;
    it.tile = local / chunks;
    const int c = local - it.tile * chunks;
    const int first = a.offsets ? __ldg(a.offsets + lo) : 0;
    const int count = (a.offsets ? __ldg(a.offsets + lo + 1) : a.rows) - first;
    const int size = (count + chunks - 1) / chunks;
    it.row0 = first + c * size;
    it.rows = min(size, count - c * size);
    return it;
}

// ---------------------------------------------------------------- weights on the lanes
//
// Tile = 128 weight rows (MMA M, TMEM lanes) x up to NT rows of x (MMA N,
// TMEM columns).  For few rows the time is that of reading the weights once:
// they go from HBM to shared memory by TMA and from there into the tensor
// cores, through no register, and the N side costs nothing where it is short.
// With SwiGLU a tile holds 64 gate rows and their 64 up rows, 16 + 16 in each
// lane quarter, so that a gate value and its up value are 16 lanes apart.
//
// 224 threads, one CTA per SM, persistent over the items:
//   warp 0     TMA producer: 128 x 128 bytes of weights and the rows' 128
//              bytes into a ring of S stages (one stage = one block of K);
//   warp 1     owns the TMEM, issues the MMAs of a stage into the next slot of
//              the accumulator ring;
//   warp 2     copies the slot's scales (xs of every row, ws) into the ring;
//   warps 3-6  add slot by slot to their sums, then write y.
// With few items K is split over a cluster: the CTAs leave their sums in
// shared memory and each finishes a share of the rows, in rank order.
template <int NT> struct Lanes;
template <> struct Lanes<32>  { static constexpr int S = 10, A = 8, BOX = 16; };
template <> struct Lanes<64>  { static constexpr int S = 8,  A = 8, BOX = 32; };
template <> struct Lanes<128> { static constexpr int S = 6,  A = 4, BOX = 32; };

constexpr int kLaneThreads = 224;

template <int NT>
struct LaneSmem {
    using L = Lanes<NT>;
    static constexpr int kWBytes = kBlock * 128;
    static constexpr int kStage = kWBytes + NT * 128;
    static constexpr int kScaleSlot = NT + 4;                     // xs of the rows, ws of gate and up
    static constexpr int kScales = L::S * kStage;
    static constexpr int kTiles = kScales + L::A * kScaleSlot * 4;
    static constexpr int kBars = kTiles + (kMaxExperts + 2) * 4;
    static constexpr int kNumBars = 2 * L::S + 3 * L::A + 1;
    static constexpr int kBytes = 1024 + kBars + 8 * kNumBars + 16;
};
static_assert(LaneSmem<32>::kBytes <= 232448 && LaneSmem<64>::kBytes <= 232448 && LaneSmem<128>::kBytes <= 232448, "smem");
static_assert(LaneSmem<32>::kBars % 8 == 0 && LaneSmem<64>::kBars % 8 == 0 && LaneSmem<128>::kBars % 8 == 0, "bars");

template <int NT, bool SWIGLU>
__global__ void __launch_bounds__(kLaneThreads, 1)
mm_lanes_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const Args a,
                int split) {
    using L = Lanes<NT>;
    using M = LaneSmem<NT>;
    constexpr int S = L::S, A = L::A;
    constexpr uint32_t kCols = NT * A;
    static_assert(kCols == 256 || kCols == 512, "TMEM columns");
    extern __shared__ uint8_t smem_dyn[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
    float* scales = reinterpret_cast<float*>(smem + M::kScales);
    int32_t* s_tiles = reinterpret_cast<int32_t*>(smem + M::kTiles);
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

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) { mbar_init(full(i), 1); mbar_init(empty(i), 1); }
        for (int i = 0; i < A; ++i) { mbar_init(acc_full(i), 1); mbar_init(acc_empty(i), 128); mbar_init(sc_full(i), 32); }
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
    count_chunks(a, NT, s_tiles);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    constexpr int kTileCols = SWIGLU ? 64 : 128;
    const int w_tiles = (a.cols + kTileCols - 1) / kTileCols;
    const int64_t items = (int64_t)min(s_tiles[a.E], a.max_chunks) * w_tiles;
    const int rank = split > 1 ? (int)cluster_rank() : 0;
    const int first = blockIdx.x / split, step = gridDim.x / split;
    const int b0 = a.kb * rank / split, b1 = a.kb * (rank + 1) / split;
    const unsigned long long limit = a.wait_limit_ns;

    if (warp == 0) {
        if (lane == 0) {
            int s = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = !a.skip_copies;
            for (int64_t i = first; ok && i < items; i += step) {
                const Item it = find_item(a, s_tiles, w_tiles, (int)i);
                const int boxes = (it.rows + L::BOX - 1) / L::BOX;
                for (int b = b0; b < b1; ++b) {
                    if (issued >= S && !(ok = mbar_wait(empty(s), ph ^ 1u, abort_flag, a.status, limit))) break;
                    const uint32_t dst = ring + s * M::kStage;
                    mbar_expect_tx(full(s), M::kWBytes + boxes * L::BOX * 128);
                    if (SWIGLU) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            tma_load_4d(dst + q * 4096, &map_w, b * kBlock, 64 * it.tile + 16 * q, 0, it.e, full(s));
                    } else {
                        tma_load_3d(dst, &map_w, b * kBlock, 128 * it.tile, it.e, full(s));
                    }
                    for (int q = 0; q < boxes; ++q)
                        tma_load_2d(dst + M::kWBytes + q * L::BOX * 128, &map_x, b * kBlock, it.row0 + q * L::BOX, full(s));
                    ++issued;
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
            }
            if (!ok) {   // let our own copies land before the CTA leaves (bounded)
                volatile uint32_t no_abort = 0;
                for (int u = max(0, issued - S); u < issued; ++u)
                    mbar_wait(full(u % S), (u / S) & 1, &no_abort, a.status, limit);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int s = 0, q = 0;
            uint32_t ph = 0, aph = 0;
            bool ok = true, wrapped = false;
            for (int64_t i = first; ok && i < items; i += step) {
                const Item it = find_item(a, s_tiles, w_tiles, (int)i);
                const uint32_t idesc = idesc_e4m3((it.rows + 15) & ~15);
                for (int b = b0; b < b1; ++b) {
                    if (wrapped && !(ok = mbar_wait(acc_empty(q), aph ^ 1u, abort_flag, a.status, limit))) break;
                    if (!(ok = mbar_wait(full(s), ph, abort_flag, a.status, limit))) break;
                    tc_fence_after();
                    const uint64_t wd = smem_desc_sw128(ring + s * M::kStage);
                    const uint64_t xd = smem_desc_sw128(ring + s * M::kStage + M::kWBytes);
#pragma unroll
                    for (int j = 0; j < 4; ++j)     // +32 bytes along K
                        mma_e4m3(tmem + q * NT, wd + 2 * j, xd + 2 * j, idesc, j != 0);
                    mma_commit(empty(s));
                    mma_commit(acc_full(q));
                    if (++s == S) { s = 0; ph ^= 1u; }
                    if (++q == A) { q = 0; aph ^= 1u; wrapped = true; }
                }
            }
            if (!ok) {   // our MMAs end before the TMEM is freed (bounded)
                volatile uint32_t no_abort = 0;
                mma_commit(drain);
                mbar_wait(drain, 0, &no_abort, a.status, limit);
            }
        }
    } else if (warp == 2) {
        int q = 0;
        uint32_t aph = 0;
        bool ok = true, wrapped = false;
        for (int64_t i = first; ok && i < items; i += step) {
            const Item it = find_item(a, s_tiles, w_tiles, (int)i);
            const float* xs = a.xs + (int64_t)it.row0 * a.kb;
            // weight rows 128 tile.. are scale row `tile`; of a gate/up weight, gate rows 64 tile.. are scale row
            // tile / 2 and their up rows n/2 further on
            const int wrow = lane == 0 ? (SWIGLU ? it.tile / 2 : it.tile) : it.tile / 2 + a.nb / 2;
            const float* ws = a.ws + ((int64_t)it.e * a.nb + wrow) * a.kb;
            for (int b = b0; b < b1; ++b) {
                if (wrapped && !(ok = warp_wait_all(acc_empty(q), aph ^ 1u, abort_flag, a.status, limit))) break;
                const uint32_t dst = smem_u32(scales + q * M::kScaleSlot);
                for (int r = lane; r < it.rows; r += 32) copy4_async(dst + 4 * r, xs + (int64_t)r * a.kb + b);
                if (lane < (SWIGLU ? 2 : 1)) copy4_async(dst + 4 * (NT + lane), ws + b);
                copies_arrive(sc_full(q));
                if (++q == A) { q = 0; aph ^= 1u; wrapped = true; }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        const int quarter = warp & 3, p = 32 * quarter + lane;
        const uint32_t lane_base = (uint32_t)(32 * quarter) << 16;
        int q = 0;
        uint32_t aph = 0;
        bool ok = true;
        for (int64_t i = first; ok && i < items; i += step) {
            const Item it = find_item(a, s_tiles, w_tiles, (int)i);
            float acc[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] = 0.f;
            for (int b = b0; b < b1; ++b) {
                if (!(ok = warp_wait_all(sc_full(q), aph, abort_flag, a.status, limit))) break;
                if (!(ok = warp_wait_all(acc_full(q), aph, abort_flag, a.status, limit))) break;
                tc_fence_after();
                const float* sc = scales + q * M::kScaleSlot;
                const float ws = sc[NT + (SWIGLU ? (lane >> 4) : 0)];
#pragma unroll
                for (int c = 0; c < NT; c += 32) {
                    if (c < it.rows) {
                        uint32_t v[32];
                        tmem_ld32(tmem + lane_base + q * NT + c, v);
                        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 x4 = *reinterpret_cast<const float4*>(sc + c + j);
                            acc[c + j] = __fmaf_rn(__uint_as_float(v[j]), x4.x * ws, acc[c + j]);
                            acc[c + j + 1] = __fmaf_rn(__uint_as_float(v[j + 1]), x4.y * ws, acc[c + j + 1]);
                            acc[c + j + 2] = __fmaf_rn(__uint_as_float(v[j + 2]), x4.z * ws, acc[c + j + 2]);
                            acc[c + j + 3] = __fmaf_rn(__uint_as_float(v[j + 3]), x4.w * ws, acc[c + j + 3]);
                        }
                    }
                }
                tc_fence_before();
                mbar_arrive(acc_empty(q));
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
            const int c = SWIGLU ? 64 * it.tile + 16 * quarter + (lane & 15) : 128 * it.tile + p;
            if (SWIGLU) {
                // lanes 0-15 hold gate rows, 16-31 their up rows; each half finishes every other row of x
#pragma unroll
                for (int t = 0; t < NT; t += 2) {
                    if (t < it.rows) {
                        const float recv = __shfl_xor_sync(0xffffffffu, lane < 16 ? acc[t + 1] : acc[t], 16);
                        const float g = lane < 16 ? acc[t] : recv, u = lane < 16 ? recv : acc[t + 1];
                        const int r = t + (lane >> 4);
                        if (r < it.rows) bq::store_value(a.y, (int64_t)(it.row0 + r) * a.ldy + c, a.ydtype, silu_f(g) * u);
                    }
                }
            } else if (c < a.cols) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (t < it.rows) bq::store_value(a.y, (int64_t)(it.row0 + t) * a.ldy + c, a.ydtype, acc[t]);
            }
        }
    }

    if (split > 1) {
        __syncwarp();
        cluster_sync();
        if (warp >= 3 && first < items && !*abort_flag) {
            const int quarter = warp & 3, p = 32 * quarter + lane;
            const Item it = find_item(a, s_tiles, w_tiles, first);
            const int c = SWIGLU ? 64 * it.tile + 16 * quarter + (lane & 15) : 128 * it.tile + p;
            for (int t = rank; t < it.rows; t += split) {
                float part[kMaxCluster];
#pragma unroll
                for (int r = 0; r < kMaxCluster; ++r)
                    part[r] = r < split ? peer_load(smem_u32(smem) + 4 * (t * 128 + p), r) : 0.f;
                float v = part[0];
#pragma unroll
                for (int r = 1; r < kMaxCluster; ++r) v += part[r];
                if (SWIGLU) {
                    const float u = __shfl_xor_sync(0xffffffffu, v, 16);
                    v = silu_f(v) * u;
                }
                if (c < a.cols && (!SWIGLU || lane < 16))
                    bq::store_value(a.y, (int64_t)(it.row0 + t) * a.ldy + c, a.ydtype, v);
            }
        }
        __syncwarp();
        cluster_sync();   // peers may still be reading this CTA's sums
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols) : "memory");
    }
}

// ---------------------------------------------------------------- rows on the lanes
//
// Tile = 128 rows of x (MMA M, TMEM lanes) x 256 weight rows (MMA N, TMEM
// columns), for many rows: there the tensor cores bound it, and with the rows
// on the lanes a block's scale is one number per thread and column half, so
// that adding a block costs one packed multiply-add per two values (against a
// scale fetched per column above).  With SwiGLU the columns are 128 gate rows
// and their 128 up rows, and a thread holds both of each.
//
// 320 threads, one CTA per SM, persistent over the items:
//   warp 0     TMA producer: 128 bytes of 128 rows and of 256 weight rows into
//              a ring of 4 stages (48 KB each);
//   warp 1     owns the TMEM (two slots of 256 columns), issues the MMAs;
//   warps 2-9  one thread per row and column half: 128 fp32 sums in registers,
//              scales read one block ahead, then y.
constexpr int kWideThreads = 320;

struct WideSmem {
    static constexpr int S = 4, A = 2, N = 256;
    static constexpr int kXBytes = 128 * 128;
    static constexpr int kStage = kXBytes + N * 128;
    static constexpr int kTiles = S * kStage;
    static constexpr int kBars = kTiles + (kMaxExperts + 2) * 4;
    static constexpr int kNumBars = 2 * S + 2 * A + 1;
    static constexpr int kBytes = 1024 + kBars + 8 * kNumBars + 16;
};
static_assert(WideSmem::kBytes <= 232448 && WideSmem::kBars % 8 == 0, "smem");

// Waits for this warp's TMEM loads; the values pass through so that no use of them moves before the wait.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                   "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                   "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
                 ::"memory");
}

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}

// acc[i] += v[2i, 2i+1] * s, sixteen pairs
__device__ __forceinline__ void add_scaled(uint64_t* acc, const uint32_t (&v)[32], uint64_t s) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        uint64_t x;
        asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "r"(v[2 * i]), "r"(v[2 * i + 1]));
        asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc[i]) : "l"(x), "l"(s));
    }
}

__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// 16 values f of a row of y from column c on: 32-byte stores where they lie in y and on 32-byte boundaries.
__device__ __forceinline__ void store16(const Args& a, int64_t row, int c, const float (&f)[16], bool wide) {
    if (wide && c + 16 <= a.cols) {
        uint8_t* p = static_cast<uint8_t*>(a.y) + (row * a.ldy + c) * (a.ydtype == BQ_DT_F32 ? 4 : 2);
        uint32_t w[8];
        if (a.ydtype == BQ_DT_F32) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(f[8 * h + i]);
                store32(p + 32 * h, w);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (a.ydtype == BQ_DT_F16) {
                w[i] = bq::h2_as_u32(__floats2half2_rn(f[2 * i], f[2 * i + 1]));
            } else {
                const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
        }
        store32(p, w);
        return;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (c + i < a.cols) bq::store_value(a.y, row * a.ldy + c + i, a.ydtype, f[i]);
}

template <bool SWIGLU>
__global__ void __launch_bounds__(kWideThreads, 1)
mm_wide_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const Args a) {
    using M = WideSmem;
    constexpr int S = M::S, A = M::A, N = M::N, kTileCols = SWIGLU ? 128 : 256;
    extern __shared__ uint8_t smem_dyn[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
    int32_t* s_tiles = reinterpret_cast<int32_t*>(smem + M::kTiles);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + M::kBars);
    const uint32_t bar0 = smem_u32(bars), ring = smem_u32(smem);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (S + s); };
    auto acc_full = [&](int q) { return bar0 + 8u * (2 * S + q); };
    auto acc_empty = [&](int q) { return bar0 + 8u * (2 * S + A + q); };
    const uint32_t drain = bar0 + 8u * (2 * S + 2 * A);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + M::kNumBars);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) { mbar_init(full(i), 1); mbar_init(empty(i), 1); }
        for (int i = 0; i < A; ++i) { mbar_init(acc_full(i), 1); mbar_init(acc_empty(i), 256); }
        mbar_init(drain, 1);
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
    count_chunks(a, 128, s_tiles);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int w_tiles = (a.cols + kTileCols - 1) / kTileCols;
    const int64_t items = (int64_t)min(s_tiles[a.E], a.max_chunks) * w_tiles;
    const unsigned long long limit = a.wait_limit_ns;

    if (warp == 0) {
        if (lane == 0) {
            int s = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = !a.skip_copies;
            for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
                const Item it = find_item(a, s_tiles, w_tiles, (int)i);
                const int boxes = (it.rows + 31) / 32;
                // the two boxes of 128 weight rows
                const int w0 = kTileCols * it.tile, w1 = SWIGLU ? a.n / 2 + w0 : w0 + 128;
                for (int b = 0; b < a.kb; ++b) {
                    if (issued >= S && !(ok = mbar_wait(empty(s), ph ^ 1u, abort_flag, a.status, limit))) break;
                    const uint32_t dst = ring + s * M::kStage;
                    mbar_expect_tx(full(s), boxes * 4096 + N * 128);
                    for (int q = 0; q < boxes; ++q)
                        tma_load_2d(dst + q * 4096, &map_x, b * kBlock, it.row0 + 32 * q, full(s));
                    tma_load_3d(dst + M::kXBytes, &map_w, b * kBlock, w0, it.e, full(s));
                    tma_load_3d(dst + M::kXBytes + 16384, &map_w, b * kBlock, w1, it.e, full(s));
                    ++issued;
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
            }
            if (!ok) {   // let our own copies land before the CTA leaves (bounded)
                volatile uint32_t no_abort = 0;
                for (int u = max(0, issued - S); u < issued; ++u)
                    mbar_wait(full(u % S), (u / S) & 1, &no_abort, a.status, limit);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = idesc_e4m3(N);
            int s = 0, q = 0;
            uint32_t ph = 0, aph = 0;
            bool ok = true, wrapped = false;
            for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
                for (int b = 0; b < a.kb; ++b) {
                    if (wrapped && !(ok = mbar_wait(acc_empty(q), aph ^ 1u, abort_flag, a.status, limit))) break;
                    if (!(ok = mbar_wait(full(s), ph, abort_flag, a.status, limit))) break;
                    tc_fence_after();
                    const uint64_t xd = smem_desc_sw128(ring + s * M::kStage);
                    const uint64_t wd = smem_desc_sw128(ring + s * M::kStage + M::kXBytes);
#pragma unroll
                    for (int j = 0; j < 4; ++j)     // +32 bytes along K
                        mma_e4m3(tmem + q * N, xd + 2 * j, wd + 2 * j, idesc, j != 0);
                    mma_commit(empty(s));
                    mma_commit(acc_full(q));
                    if (++s == S) { s = 0; ph ^= 1u; }
                    if (++q == A) { q = 0; aph ^= 1u; wrapped = true; }
                }
            }
            if (!ok) {   // our MMAs end before the TMEM is freed (bounded)
                volatile uint32_t no_abort = 0;
                mma_commit(drain);
                mbar_wait(drain, 0, &no_abort, a.status, limit);
            }
        }
    } else {
        const int quarter = warp & 3, half = (warp - 2) >> 2, p = 32 * quarter + lane;
        // this thread's columns: 64 from c_lo on and 64 from c_hi on (with SwiGLU gate columns and their up columns)
        const uint32_t c_lo = SWIGLU ? 64 * half : 128 * half, c_hi = SWIGLU ? 128 + 64 * half : 128 * half + 64;
        const uint32_t base = tmem + ((uint32_t)(32 * quarter) << 16);
        const int es = a.ydtype == BQ_DT_F32 ? 4 : 2;
        const bool wide = (reinterpret_cast<uintptr_t>(a.y) | (uintptr_t)(a.ldy * es)) % 32 == 0;
        int q = 0;
        uint32_t aph = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const Item it = find_item(a, s_tiles, w_tiles, (int)i);
            const float* xs = a.xs + (int64_t)(it.row0 + min(p, it.rows - 1)) * a.kb;
            const int wb_lo = SWIGLU ? it.tile : min(2 * it.tile + half, a.nb - 1);
            const float* ws_lo = a.ws + ((int64_t)it.e * a.nb + wb_lo) * a.kb;
            const float* ws_hi = SWIGLU ? ws_lo + (int64_t)(a.nb / 2) * a.kb : ws_lo;
            uint64_t acc[64];
#pragma unroll
            for (int j = 0; j < 64; ++j) acc[j] = 0ull;
            float x_next = __ldg(xs), lo_next = __ldg(ws_lo), hi_next = SWIGLU ? __ldg(ws_hi) : 0.f;
            for (int b = 0; b < a.kb; ++b) {
                const float s_lo = x_next * lo_next, s_hi = SWIGLU ? x_next * hi_next : s_lo;
                const uint64_t lo2 = pack2(s_lo, s_lo), hi2 = pack2(s_hi, s_hi);
                const int bn = min(b + 1, a.kb - 1);
                x_next = __ldg(xs + bn);
                lo_next = __ldg(ws_lo + bn);
                if (SWIGLU) hi_next = __ldg(ws_hi + bn);
                if (!(ok = warp_wait_all(acc_full(q), aph, abort_flag, a.status, limit))) break;
                tc_fence_after();
                uint32_t v0[32], v1[32];
                const uint32_t t = base + q * N;
                tmem_ld32(t + c_lo, v0);
                tmem_wait_ld(v0);
                tmem_ld32(t + c_lo + 32, v1);
                add_scaled(acc, v0, lo2);
                tmem_wait_ld(v1);
                tmem_ld32(t + c_hi, v0);
                add_scaled(acc + 16, v1, lo2);
                tmem_wait_ld(v0);
                tmem_ld32(t + c_hi + 32, v1);
                add_scaled(acc + 32, v0, hi2);
                tmem_wait_ld(v1);
                tc_fence_before();
                mbar_arrive(acc_empty(q));
                add_scaled(acc + 48, v1, hi2);
                if (++q == A) { q = 0; aph ^= 1u; }
            }
            if (!ok) break;
            if (p < it.rows) {
                const int c0 = kTileCols * it.tile + (SWIGLU ? 64 : 128) * half;
#pragma unroll
                for (int g = 0; g < (SWIGLU ? 4 : 8); ++g) {
                    float f[16];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 v = unpack2(acc[8 * g + j]);
                        f[2 * j] = v.x;
                        f[2 * j + 1] = v.y;
                        if (SWIGLU) {
                            const float2 u = unpack2(acc[32 + ((8 * g + j) & 31)]);
                            f[2 * j] = silu_f(v.x) * u.x;
                            f[2 * j + 1] = silu_f(v.y) * u.y;
                        }
                    }
                    store16(a, it.row0 + p, c0 + 16 * g, f, wide);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
}

// ---------------------------------------------------------------- host side
bool encode(CUtensorMap* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
            const uint32_t* box) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), dims, strides, box, ones,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows [rows][k] in boxes of 128 bytes x `box` rows.
bool row_map(CUtensorMap* map, const uint8_t* x, int rows, int k, int box) {
    const uint64_t dims[2] = {(uint64_t)k, (uint64_t)rows}, strides[1] = {(uint64_t)k};
    const uint32_t b[2] = {kBlock, (uint32_t)box};
    return encode(map, x, 2, dims, strides, b);
}

// Weights [E][n][k] in boxes of 128 bytes x 128 rows; of a gate/up weight
// [E][2][n/2][k] in boxes of 16 gate rows and their 16 up rows.
bool weight_map(CUtensorMap* map, const uint8_t* w, int E, int n, int k, bool swiglu) {
    if (!swiglu) {
        const uint64_t dims[3] = {(uint64_t)k, (uint64_t)n, (uint64_t)E}, strides[2] = {(uint64_t)k, (uint64_t)n * k};
        const uint32_t b[3] = {kBlock, 128, 1};
        return encode(map, w, 3, dims, strides, b);
    }
    const uint64_t h = n / 2;
    const uint64_t dims[4] = {(uint64_t)k, h, 2, (uint64_t)E}, strides[3] = {(uint64_t)k, h * k, (uint64_t)n * k};
    const uint32_t b[4] = {kBlock, 16, 2, 1};
    return encode(map, w, 4, dims, strides, b);
}

constexpr int kSms = 152;

template <int NT, bool SWIGLU>
cudaError_t launch_lanes(const CUtensorMap& map_w, const CUtensorMap& map_x, const Args& a, int64_t items, int split,
                         cudaStream_t st) {
    // per device: the attribute is a property of the function on the current device
    static std::atomic<bool> attr_set[64];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_set[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(mm_lanes_kernel<NT, SWIGLU>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   LaneSmem<NT>::kBytes);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(split > 1 ? items * split : std::min<int64_t>(items, kSms)));
    cfg.blockDim = dim3(kLaneThreads);
    cfg.dynamicSmemBytes = LaneSmem<NT>::kBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, mm_lanes_kernel<NT, SWIGLU>, map_w, map_x, a, split);
}

template <bool SWIGLU>
cudaError_t launch_wide(const CUtensorMap& map_w, const CUtensorMap& map_x, const Args& a, int64_t items,
                        cudaStream_t st) {
    static std::atomic<bool> attr_set[64];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_set[dev].load(std::memory_order_acquire)) {
        const cudaError_t e =
            cudaFuncSetAttribute(mm_wide_kernel<SWIGLU>, cudaFuncAttributeMaxDynamicSharedMemorySize, WideSmem::kBytes);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(true, std::memory_order_release);
    }
    return bq::launch_after(mm_wide_kernel<SWIGLU>, dim3((unsigned)std::min<int64_t>(items, kSms)), dim3(kWideThreads),
                            WideSmem::kBytes, st, map_w, map_x, a);
}

bq_status run_mm(const char* name, const uint8_t* x, const float* xscales, int32_t rows, const int32_t* offsets,
                 int32_t E, const uint8_t* w, const float* wscales, int32_t n, int32_t k, int32_t swiglu, void* y,
                 int32_t ydtype, int64_t ldy, cudaStream_t st) {
    const int es = bq::dtype_size(ydtype);
    if (es == 0) return bq::fail(BQ_ERR_FORMAT, "%s: unknown element type %d", name, ydtype);
    if (swiglu != 0 && swiglu != 1) return bq::fail(BQ_ERR_SHAPE, "%s: swiglu must be 0 or 1, not %d", name, swiglu);
    if (rows < 0 || n < 1 || k < 16 || k % 16)
        return bq::fail(BQ_ERR_SHAPE, "%s: %d rows, n = %d, k = %d (k must be a positive multiple of 16)", name, rows,
                        n, k);
    if (swiglu && n % 256)
        return bq::fail(BQ_ERR_SHAPE, "%s: a gate/up weight needs n = %d to be a multiple of 256", name, n);
    if (E < 1 || E > kMaxExperts || (int64_t)E * n > (int64_t)INT32_MAX)
        return bq::fail(BQ_ERR_SHAPE, "%s: E = %d outside [1, 1024], or E * n beyond %d", name, E, INT32_MAX);
    if (rows == 0) return BQ_OK;
    if (!x || !xscales || !w || !wscales || !y) return bq::fail(BQ_ERR_NULL, "%s: NULL pointer", name);
    const int cols = swiglu ? n / 2 : n;
    if (ldy < cols)
        return bq::fail(BQ_ERR_SHAPE, "%s: rows of y are %lld elements apart, fewer than their %d", name,
                        (long long)ldy, cols);
    if (!bq::aligned(x, 16) || !bq::aligned(w, 16) || !bq::aligned(xscales, 4) || !bq::aligned(wscales, 4) ||
        !bq::aligned(offsets, 4) || !bq::aligned(y, es))
        return bq::fail(BQ_ERR_ALIGN, "%s: x and w must be 16-byte aligned, scales and offsets 4-byte, y to its element",
                        name);
    const int experts = offsets ? std::min(E, rows) : 1;   // that can have rows
    // most row chunks and items there can be, for the grid and (as an int) inside the kernel
    auto chunks_of = [&](int most) { return (int64_t)(rows + most - 1) / most + (offsets ? experts : 0); };
    auto tiles_of = [&](int width) { return (int64_t)(cols + width - 1) / width; };
    const bool wide = rows / experts >= 96 && chunks_of(128) * tiles_of(swiglu ? 128 : 256) >= 100;
    const int nt = rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
    const int64_t chunks = chunks_of(wide ? 128 : nt);
    const int64_t items = chunks * (wide ? tiles_of(swiglu ? 128 : 256) : tiles_of(swiglu ? 64 : 128));
    if (items > INT32_MAX / 2) return bq::fail(BQ_ERR_SHAPE, "%s: %d rows x %d columns are too many", name, rows, cols);
    bq_status s = bq::check_arch();
    if (s != BQ_OK) return s;
    const bq::WaitProbe probe = bq::wait_probe();
    const Args a{xscales, rows, offsets, E, wscales, n, k, (k + kBlock - 1) / kBlock, (n + kBlock - 1) / kBlock, cols,
                 y, ydtype, ldy, bq::device_status_ptr(), probe.limit_ns, probe.skip_weight_copies, (int)chunks};
    CUtensorMap map_w, map_x;
    if (!weight_map(&map_w, w, E, n, k, swiglu && !wide) || !row_map(&map_x, x, rows, k, !wide && nt == 32 ? 16 : 32))
        return bq::fail(BQ_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", name);
    cudaError_t e;
    if (wide) {
        e = swiglu ? launch_wide<true>(map_w, map_x, a, items, st) : launch_wide<false>(map_w, map_x, a, items, st);
    } else {
        int split = 1;
        while (split < kMaxCluster && items * split * 2 <= kSms && a.kb >= 4 * split) split *= 2;
        auto go = [&](auto width) {
            constexpr int NT = decltype(width)::value;
            return swiglu ? launch_lanes<NT, true>(map_w, map_x, a, items, split, st)
                          : launch_lanes<NT, false>(map_w, map_x, a, items, split, st);
        };
        e = nt == 32 ? go(std::integral_constant<int, 32>()) : nt == 64 ? go(std::integral_constant<int, 64>())
                                                                          : go(std::integral_constant<int, 128>());
    }
    if (e != cudaSuccess) return bq::fail(BQ_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
    bq::note_launch();
    return bq::check_launch(name);
}

}  // namespace

extern "C" bq_status bq_mm_fp8_b128(const uint8_t* x, const float* xscales, int32_t m, const uint8_t* w,
                                    const float* wscales, int32_t n, int32_t k, int32_t swiglu, void* y,
                                    int32_t ydtype, int64_t ldy, bq_stream_t stream) {
    return run_mm("bq_mm_fp8_b128", x, xscales, m, nullptr, 1, w, wscales, n, k, swiglu, y, ydtype, ldy,
                  (cudaStream_t)stream);
}

extern "C" bq_status bq_moe_mm_fp8_b128(const uint8_t* x, const float* xscales, int32_t rows, const int32_t* offsets,
                                        int32_t E, const uint8_t* w, const float* wscales, int32_t n, int32_t k,
                                        int32_t swiglu, void* y, int32_t ydtype, int64_t ldy, bq_stream_t stream) {
    if (rows > 0 && !offsets) return bq::fail(BQ_ERR_NULL, "bq_moe_mm_fp8_b128: offsets is NULL");
    return run_mm("bq_moe_mm_fp8_b128", x, xscales, rows, offsets, E, w, wscales, n, k, swiglu, y, ydtype, ldy,
                  (cudaStream_t)stream);
}
