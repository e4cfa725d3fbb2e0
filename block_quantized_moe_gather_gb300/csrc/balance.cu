// What trains a router: the balance loss and z-loss of its logits with the
// per-expert counts, and the gradient of router weights and of both losses
// with respect to the logits.
//
// With z = logits + bias, m = max z, S = sum exp(z - m), lse = m + log S:
//   softmax rules    p_e = exp(z_e - m) / S
//   score rule       p_e = s_e / sum s,  s = sqrt(softplus(z))
// and per sequence of n rows, c_e its pairs of expert e, P_e its mean p_e:
//   balance = mean over sequences of sum_e (E c_e / (k n)) P_e,  z-loss = mean over rows of lse^2.
// Gradients, with a_e = dbalance E c_e / (k n) / (n sequences) and w the router weights of the k selected:
//   softmax rules    dz = p (a - <p, a>)               + 2 dz-loss lse p / rows;  selected: + w (dw - <w, dw>)
//   score rule       dz = s' (a - <p, a>) / sum s      + 2 dz-loss lse softmax / rows;  selected: + scale s' dw
//                    s' = sigmoid(z) / (2 s)
#include <algorithm>

#include "row_types.cuh"

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSequences = 65536;

enum { RULE_SOFTMAX = 0, RULE_SCORE = 1 };

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int off = 16; off; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// sqrt(softplus(z)); below -20 softplus is exp(z) to 1e-9, and its root exp(z / 2) stays normal where exp(z) does not.
__device__ __forceinline__ float score_of(float z) {
    return z < -20.f ? expf(0.5f * z) : sqrtf(fmaxf(z, 0.f) + log1pf(expf(-fabsf(z))));
}

// Its derivative, sigmoid(z) / (2 score).
__device__ __forceinline__ float score_slope(float z, float score) {
    return z < -20.f ? 0.5f * score : 0.5f / ((1.f + expf(-z)) * score);
}

// A row of logits in a warp: lane l holds experts l + 32 i (z; -inf behind the last).
template <int NPER>
__device__ __forceinline__ void load_row(const float* row, const float* bias, int E, int lane, float (&z)[NPER]) {
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
        const int e = lane + 32 * i;
        z[i] = e < E ? __ldg(row + e) : -INFINITY;
    }
    if (bias) {
#pragma unroll
        for (int i = 0; i < NPER; ++i)
            if (lane + 32 * i < E) z[i] = __fadd_rn(z[i], __ldg(bias + lane + 32 * i));
    }
}

// Softmax and log-sum-exp of a row.  A row of -inf only has probabilities 0 and a log-sum-exp counted as 0.
template <int NPER>
__device__ __forceinline__ void softmax_row(const float (&z)[NPER], float (&p)[NPER], float& lse) {
    float m = z[0];
#pragma unroll
    for (int i = 1; i < NPER; ++i) m = fmaxf(m, z[i]);
    m = warp_max(m);
    if (m == -INFINITY) m = 0.f;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
        p[i] = expf(z[i] - m);
        sum += p[i];
    }
    sum = warp_sum(sum);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    lse = sum == 0.f ? 0.f : m + logf(sum);
#pragma unroll
    for (int i = 0; i < NPER; ++i) p[i] *= inv;
}

// Scores over their sum, and 1 / the sum (0 where every score is).
template <int NPER>
__device__ __forceinline__ void score_row(const float (&z)[NPER], int E, int lane, float (&s)[NPER], float& inv) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
        s[i] = lane + 32 * i < E ? score_of(z[i]) : 0.f;
        sum += s[i];
    }
    sum = warp_sum(sum);
    inv = sum == 0.f ? 0.f : 1.f / sum;
}

// ---------------------------------------------------------------- sequences
// Sequence s of `offsets` [S + 1], or all T rows where there are none; false (and recorded) if it is no range of [0, T].
__device__ __forceinline__ bool sequence(const int32_t* offsets, int s, int T, int32_t* status, int& lo, int& hi) {
    lo = offsets ? __ldg(offsets + s) : 0;
    hi = offsets ? __ldg(offsets + s + 1) : T;
    if (0 <= lo && lo <= hi && hi <= T) return true;
    bq::set_device_error(status, BQ_DEV_BAD_ROW);
    hi = lo;
    return false;
}

// Sequences that have rows, and their rows (all threads; contains barriers).
__device__ __forceinline__ void sequence_totals(const int32_t* offsets, int S, int T, int32_t* status, int* s_totals) {
    if (threadIdx.x < 2) s_totals[threadIdx.x] = 0;
    __syncthreads();
    int used = 0, rows = 0;
    for (int s = threadIdx.x; s < S; s += blockDim.x) {
        int lo, hi;
        if (sequence(offsets, s, T, status, lo, hi) && hi > lo) { ++used; rows += hi - lo; }
    }
    if (used) {
        atomicAdd(&s_totals[0], used);
        atomicAdd(&s_totals[1], rows);
    }
    __syncthreads();
}

// First sequence that ends behind `row` (all threads of the CTA; contains barriers).
__device__ __forceinline__ int first_sequence(const int32_t* offsets, int S, int row) {
    int n = 0;
    if (offsets)
        for (int s = threadIdx.x; s - (int)threadIdx.x < S; s += blockDim.x)
            n += __syncthreads_count(s < S && __ldg(offsets + s + 1) <= row);
    return n;
}

// ---------------------------------------------------------------- counts, mean probabilities, losses
struct BalanceArgs {
    const float* logits;
    const float* bias;
    int T, E, k;
    const int32_t* ids;
    const int32_t* offsets;
    int S;
    int chunk_rows, chunks;
    float* part_p;       // [chunks + S][E]
    int32_t* part_c;     // [chunks + S][E]
    float* part_z;       // [chunks + S]
    int32_t* counts;
    float* probs;
    float* losses;
    int32_t* status;
};

// The rows are cut into chunks of equal size, a CTA each, whatever sequences they belong to: one long sequence among
// short ones takes no longer than many of equal length.  Chunk c leaves its sums over sequence s in slot c + s: along
// rows that ascend, either c or s grows from one (chunk, sequence) to the next, so no two share a slot.
template <int NPER, int RULE>
__device__ __forceinline__ void chunk_sums(const BalanceArgs& a, float* s_red, int32_t* s_hist) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t first = (int64_t)blockIdx.x * a.chunk_rows;
    const int row0 = (int)first, row1 = (int)min((int64_t)a.T, first + a.chunk_rows);
    for (int s = first_sequence(a.offsets, a.S, row0); s < a.S; ++s) {
        int lo, hi;
        sequence(a.offsets, s, a.T, a.status, lo, hi);
        if (lo >= row1) break;
        lo = max(lo, row0);
        hi = min(hi, row1);
        if (lo >= hi) continue;
        for (int e = threadIdx.x; e < a.E; e += kThreads) s_hist[e] = 0;
        __syncthreads();
        for (int64_t i = (int64_t)lo * a.k + threadIdx.x; i < (int64_t)hi * a.k; i += kThreads) {
            const int e = __ldg(a.ids + i);
            if (e >= 0 && e < a.E) atomicAdd(&s_hist[e], 1);
            else bq::set_device_error(a.status, BQ_DEV_BAD_EXPERT_ID);
        }
        float acc[NPER], z2 = 0.f;
#pragma unroll
        for (int i = 0; i < NPER; ++i) acc[i] = 0.f;
        for (int r = lo + warp; r < hi; r += kWarps) {
            float z[NPER], p[NPER], lse, inv = 1.f;
            load_row(a.logits + (int64_t)r * a.E, a.bias, a.E, lane, z);
            softmax_row(z, p, lse);
            if (RULE == RULE_SCORE) score_row(z, a.E, lane, p, inv);
#pragma unroll
            for (int i = 0; i < NPER; ++i) acc[i] = __fmaf_rn(p[i], inv, acc[i]);
            z2 = __fmaf_rn(lse, lse, z2);
        }
#pragma unroll
        for (int i = 0; i < NPER; ++i)
            if (lane + 32 * i < a.E) s_red[warp * a.E + lane + 32 * i] = acc[i];
        if (lane == 0) s_red[kWarps * a.E + warp] = z2;
        __syncthreads();
        const int64_t slot = (int64_t)blockIdx.x + s;
        for (int e = threadIdx.x; e < a.E; e += kThreads) {
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) sum += s_red[w * a.E + e];
            a.part_p[slot * a.E + e] = sum;
            a.part_c[slot * a.E + e] = s_hist[e];
        }
        if (threadIdx.x == 0) {
            float sum = 0.f;
            for (int w = 0; w < kWarps; ++w) sum += s_red[kWarps * a.E + w];
            a.part_z[slot] = sum;
        }
        __syncthreads();
    }
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

// The slots of every sequence added up, by the CTAs of one cluster.  A group is 32 experts of a sequence; `share` warps
// (a power of two) take a share of its slots each.
__device__ __forceinline__ void finish(const BalanceArgs& a, int rank, int ranks, int share, float* s_red, int32_t* s_redc) {
    __shared__ int s_totals[2];
    __shared__ float s_loss[2][kWarps];
    __shared__ float s_cta[2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    sequence_totals(a.offsets, a.S, a.T, a.status, s_totals);
    const int blocks = (a.E + 31) / 32, sub = warp & (share - 1), at_once = kWarps / share;
    const int64_t groups = (int64_t)a.S * blocks;
    float balance = 0.f, z2 = 0.f;
    for (int64_t g0 = (int64_t)rank * at_once; g0 < groups; g0 += (int64_t)ranks * at_once) {
        const int64_t g = g0 + warp / share;
        const int s = (int)(g / blocks), block = (int)(g - (int64_t)s * blocks), e = block * 32 + lane;
        int lo = 0, hi = 0;
        if (g < groups) sequence(a.offsets, s, a.T, a.status, lo, hi);
        float p = 0.f;
        int c = 0;
        if (hi > lo) {
            const int64_t begin = lo / a.chunk_rows + (int64_t)s, end = (hi - 1) / a.chunk_rows + (int64_t)s + 1;
            if (e < a.E) {
#pragma unroll 8
                for (int64_t i = begin + sub; i < end; i += share) {
                    p += a.part_p[i * a.E + e];
                    c += a.part_c[i * a.E + e];
                }
            }
            if (block == 0)
                for (int64_t i = begin + 32 * sub + lane; i < end; i += 32 * share) z2 += a.part_z[i];
        }
        if (share > 1) {
            s_red[threadIdx.x] = p;
            s_redc[threadIdx.x] = c;
            __syncthreads();
            if (sub == 0) {
                for (int w = 1; w < share; ++w) {
                    p += s_red[threadIdx.x + 32 * w];
                    c += s_redc[threadIdx.x + 32 * w];
                }
            }
            __syncthreads();
        }
        if (sub == 0 && g < groups && e < a.E) {
            const float n = (float)(hi - lo), mean = hi > lo ? p / n : 0.f;
            a.counts[(int64_t)s * a.E + e] = c;
            a.probs[(int64_t)s * a.E + e] = mean;
            if (hi > lo) balance += (float)c * ((float)a.E / ((float)a.k * n)) * mean;
        }
    }
    balance = warp_sum(balance);
    z2 = warp_sum(z2);
    if (lane == 0) { s_loss[0][warp] = balance; s_loss[1][warp] = z2; }
    __syncthreads();
    if (threadIdx.x < 2) {
        float v = 0.f;
        for (int w = 0; w < kWarps; ++w) v += s_loss[threadIdx.x][w];
        s_cta[threadIdx.x] = v;
    }
    if (ranks > 1) cluster_sync();
    else __syncthreads();
    if (rank == 0 && threadIdx.x < 2) {
        float v = 0.f;
        for (int r = 0; r < ranks; ++r) v += ranks > 1 ? peer_load(&s_cta[threadIdx.x], r) : s_cta[threadIdx.x];
        const int n = s_totals[threadIdx.x];
        a.losses[threadIdx.x] = n ? v / (float)n : 0.f;
    }
    if (ranks > 1) cluster_sync();   // rank 0 may still be reading
}

__device__ __forceinline__ int cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return (int)r;
}

// Shared memory, in 4-byte words: kWarps rows of E sums and their z sums, then E counts; at least a word of each per
// thread, which is what finish() takes.
__host__ __device__ inline int sums_words(int E) { return kWarps * E + kWarps > kThreads ? kWarps * E + kWarps : kThreads; }
inline size_t balance_smem(int E) { return ((size_t)sums_words(E) + std::max(E, kThreads)) * 4; }

// ONE: the launch is one cluster, which also adds its slots up.
template <int NPER, int RULE, bool ONE>
__global__ void __launch_bounds__(kThreads)
balance_kernel(const BalanceArgs a, int share) {
    extern __shared__ float s_dyn[];
    bq::grid_dependency_wait();   // launched behind whatever precedes it on the stream
    bq::allow_dependents();
    int32_t* hist = reinterpret_cast<int32_t*>(s_dyn + sums_words(a.E));
    chunk_sums<NPER, RULE>(a, s_dyn, hist);
    if (ONE) {
        const int ranks = gridDim.x;
        if (ranks > 1) cluster_sync();   // the slots that the others wrote
        else __syncthreads();
        finish(a, ranks > 1 ? cluster_rank() : 0, ranks, share, s_dyn, hist);
    }
}

__global__ void __launch_bounds__(kThreads)
balance_finish_kernel(const BalanceArgs a, int share) {
    __shared__ float s_red[kThreads];
    __shared__ int32_t s_redc[kThreads];
    bq::grid_dependency_wait();
    bq::allow_dependents();
    finish(a, cluster_rank(), gridDim.x, share, s_red, s_redc);
}

// ---------------------------------------------------------------- gradient
struct RouteGradArgs {
    const float* logits;
    const float* bias;
    int T, E, k;
    const int32_t* ids;
    const float* dweights;   // or NULL
    float scale;
    const int32_t* counts;   // [S][E], with losses
    const float* dlosses;    // [2], or NULL
    const int32_t* offsets;
    int S;
    int chunk_rows;
    void* dlogits;
    int dtype;
    float* part_b;           // [chunks][E] sums of the bias gradient, or NULL
    int32_t* status;
};

// A warp per row, the whole gradient of the row in its registers: logits are read once, gradients written once.
template <int NPER, int RULE, bool LOSSES>
__global__ void __launch_bounds__(kThreads)
route_backward_kernel(const RouteGradArgs a) {
    extern __shared__ float s_dyn[];
    __shared__ int s_totals[2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    bq::grid_dependency_wait();   // launched behind whatever precedes it on the stream
    bq::allow_dependents();
    const int64_t first = (int64_t)blockIdx.x * a.chunk_rows;
    const int row0 = (int)first, row1 = (int)min((int64_t)a.T, first + a.chunk_rows);
    float per_seq = 0.f, per_row = 0.f;
    if (LOSSES) {
        sequence_totals(a.offsets, a.S, a.T, a.status, s_totals);
        per_seq = __ldg(a.dlosses) * ((float)a.E / (float)a.k) / (float)max(1, s_totals[0]);
        per_row = 2.f * __ldg(a.dlosses + 1) / (float)max(1, s_totals[1]);
    }
    int s = first_sequence(a.offsets, a.S, row0), lo = 0, hi = a.T;
    if (a.offsets) lo = hi = -1;
    float acc[NPER], weight[NPER];
#pragma unroll
    for (int i = 0; i < NPER; ++i) acc[i] = weight[i] = 0.f;
    bool fresh = true;
    for (int r = row0 + warp; r < row1; r += kWarps) {
        if (a.offsets) {   // rows ascend, so the sequences do too; rows in none are left out
            while (s < a.S && r >= hi) {
                sequence(a.offsets, s, a.T, a.status, lo, hi);
                fresh = true;
                if (r >= hi) ++s;
            }
            if (r < lo || r >= hi) continue;
        }
        if (LOSSES && fresh) {
            const float n = (float)(hi - lo);
#pragma unroll
            for (int i = 0; i < NPER; ++i) {
                const int e = lane + 32 * i;
                weight[i] = e < a.E ? (float)__ldg(a.counts + (int64_t)s * a.E + e) * (per_seq / n / n) : 0.f;
            }
            fresh = false;
        }
        const float* row = a.logits + (int64_t)r * a.E;
        // the selected experts, a lane each: their logit, weight and the gradient that the weights bring
        int id = -1;
        float dw = 0.f, zs = -INFINITY;
        if (a.dweights && lane < a.k) {
            id = __ldg(a.ids + (int64_t)r * a.k + lane);
            if (id < 0 || id >= a.E) {
                bq::set_device_error(a.status, BQ_DEV_BAD_EXPERT_ID);
                id = -1;
            } else {
                dw = __ldg(a.dweights + (int64_t)r * a.k + lane);
                zs = __ldg(row + id);
                if (a.bias) zs = __fadd_rn(zs, __ldg(a.bias + id));
            }
        }
        float d[NPER];
#pragma unroll
        for (int i = 0; i < NPER; ++i) d[i] = 0.f;
        if (LOSSES) {
            float z[NPER], p[NPER], lse;
            load_row(row, a.bias, a.E, lane, z);
            softmax_row(z, p, lse);
            const float f = per_row * lse;
            if (RULE == RULE_SOFTMAX) {
                float dot = 0.f;
#pragma unroll
                for (int i = 0; i < NPER; ++i) dot = __fmaf_rn(p[i], weight[i], dot);
                dot = warp_sum(dot);
#pragma unroll
                for (int i = 0; i < NPER; ++i) d[i] = p[i] * (weight[i] - dot + f);
            } else {
                float sc[NPER], inv, dot = 0.f;
                score_row(z, a.E, lane, sc, inv);
#pragma unroll
                for (int i = 0; i < NPER; ++i) dot = __fmaf_rn(sc[i] * inv, weight[i], dot);
                dot = warp_sum(dot);
#pragma unroll
                for (int i = 0; i < NPER; ++i) {
                    const float t = sc[i] == 0.f ? 0.f : score_slope(z[i], sc[i]) * inv * (weight[i] - dot);
                    d[i] = __fmaf_rn(p[i], f, t);
                }
            }
        }
        if (a.dweights) {
            float g;
            if (RULE == RULE_SOFTMAX) {
                const float m = warp_max(zs);
                const float ex = id >= 0 ? expf(zs - m) : 0.f;
                const float w = ex / warp_sum(ex);
                const float mean = warp_sum(id >= 0 ? w * dw : 0.f);
                g = w * (dw - mean);
            } else {
                const float sc = score_of(zs);
                g = id >= 0 && sc != 0.f ? a.scale * dw * score_slope(zs, sc) : 0.f;
            }
            for (int j = 0; j < a.k; ++j) {
                const int ej = __shfl_sync(0xffffffffu, id, j);
                const float gj = __shfl_sync(0xffffffffu, g, j);
                if (ej >= 0 && (ej & 31) == lane) {
#pragma unroll
                    for (int i = 0; i < NPER; ++i)
                        if (ej >> 5 == i) d[i] += gj;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NPER; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E) bq::store_value(a.dlogits, (int64_t)r * a.E + e, a.dtype, d[i]);
            acc[i] += d[i];
        }
    }
    if (!a.part_b) return;
#pragma unroll
    for (int i = 0; i < NPER; ++i)
        if (lane + 32 * i < a.E) s_dyn[warp * a.E + lane + 32 * i] = acc[i];
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += s_dyn[w * a.E + e];
        a.part_b[(int64_t)blockIdx.x * a.E + e] = sum;
    }
}

// out[e] = the sum of part[0..parts)[e], 32 columns a CTA.
__global__ void __launch_bounds__(kThreads)
column_sums_kernel(const float* part, int parts, int cols, float* out) {
    __shared__ float s_red[kWarps][32];
    bq::grid_dependency_wait();
    bq::allow_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
    float sum = 0.f;
    if (e < cols) {
#pragma unroll 4
        for (int i = warp; i < parts; i += kWarps) sum += part[(int64_t)i * cols + e];
    }
    s_red[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && e < cols) {
        for (int w = 1; w < kWarps; ++w) sum += s_red[w][lane];
        out[e] = sum;
    }
}

// ---------------------------------------------------------------- host side
constexpr int kSms = 152;

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// Rows of a chunk and the number of chunks.
struct Chunking {
    int rows, chunks;
};

Chunking chunking(int T, int most, int least) {
    const int rows = std::max(least, (int)(((int64_t)T + most - 1) / most));
    return {rows, (int)(((int64_t)T + rows - 1) / rows)};
}

constexpr int kOneClusterRows = 1024;

Chunking balance_chunking(int T) { return T <= kOneClusterRows ? chunking(T, 8, kWarps) : chunking(T, 2 * kSms, kWarps); }

Chunking gradient_chunking(int T) { return chunking(T, 2 * kSms, kWarps); }

template <typename F>
void with_nper(int E, F f) {
    if (E <= 32) f(std::integral_constant<int, 1>());
    else if (E <= 64) f(std::integral_constant<int, 2>());
    else if (E <= 128) f(std::integral_constant<int, 4>());
    else if (E <= 256) f(std::integral_constant<int, 8>());
    else if (E <= 512) f(std::integral_constant<int, 16>());
    else f(std::integral_constant<int, 32>());
}

bq_status check_router(const char* name, int T, int E, int k, int scoring, const int32_t* offsets, int S) {
    if (T < 0) return bq::fail(BQ_ERR_SHAPE, "%s: T = %d < 0", name, T);
    if (E < 1 || E > 1024) return bq::fail(BQ_ERR_SHAPE, "%s: E = %d outside [1, 1024]", name, E);
    if (k < 1 || k > 8 || k > E) return bq::fail(BQ_ERR_SHAPE, "%s: k = %d outside [1, min(8, E)]", name, k);
    if ((int64_t)T * k > (int64_t)INT32_MAX)
        return bq::fail(BQ_ERR_SHAPE, "%s: T * k = %lld pairs exceeds %d", name, (long long)T * k, INT32_MAX);
    if (scoring < BQ_SCORE_SOFTMAX || scoring > BQ_SCORE_SQRTSOFTPLUS)
        return bq::fail(BQ_ERR_SHAPE, "%s: unknown scoring rule %d", name, scoring);
    if (S < 1 || S > kMaxSequences || (!offsets && S != 1))
        return bq::fail(BQ_ERR_SHAPE, "%s: %d sequences (1 without offsets, at most %d with)", name, S, kMaxSequences);
    return BQ_OK;
}

bq_status check4(const char* name, const char* what, const void* p, bool needed) {
    if (needed && !p) return bq::fail(BQ_ERR_NULL, "%s: %s is NULL", name, what);
    if (!bq::aligned(p, 4)) return bq::fail(BQ_ERR_ALIGN, "%s: %s must be 4-byte aligned", name, what);
    return BQ_OK;
}

bq_status launched(const char* name, cudaError_t e) {
    if (e != cudaSuccess) {
        cudaGetLastError();   // reported here
        return bq::fail(BQ_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
    }
    bq::note_launch();
    return bq::check_launch(name);
}

// Launch behind the stream's last kernel, as one cluster of all its CTAs.
template <typename Kernel, typename... Args>
cudaError_t launch_cluster(Kernel kernel, int ctas, size_t smem, cudaStream_t st, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename Kernel>
cudaError_t allow_smem(Kernel kernel, size_t smem) {
    return smem <= 48 * 1024 ? cudaSuccess
                             : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
}

// Warps that share a group of experts: enough for about four slots each.
int share_of(int64_t slots, int S) {
    int share = 1;
    while (share < kWarps && slots / S > 4 * share) share *= 2;
    return share;
}

}  // namespace

extern "C" size_t bq_moe_balance_workspace_bytes(int32_t T, int32_t E, int32_t S) {
    if (T < 0 || E < 1 || E > 1024 || S < 1 || S > kMaxSequences) return 0;
    const size_t slots = (size_t)balance_chunking(T).chunks + S;
    return 2 * up256(slots * E * 4) + up256(slots * 4);
}

extern "C" bq_status bq_moe_balance_loss(const float* logits, const float* bias, int32_t T, int32_t E,
                                         const int32_t* ids, int32_t k, int32_t scoring, const int32_t* seq_offsets,
                                         int32_t S, int32_t* counts, float* probs, float* losses, void* workspace,
                                         size_t workspace_bytes, bq_stream_t stream) {
    const char* name = "bq_moe_balance_loss";
    bq_status s = check_router(name, T, E, k, scoring, seq_offsets, S);
    if (s != BQ_OK || (s = check4(name, "logits", logits, T > 0)) != BQ_OK ||
        (s = check4(name, "bias", bias, false)) != BQ_OK || (s = check4(name, "ids", ids, T > 0)) != BQ_OK ||
        (s = check4(name, "seq_offsets", seq_offsets, false)) != BQ_OK ||
        (s = check4(name, "counts", counts, true)) != BQ_OK || (s = check4(name, "probs", probs, true)) != BQ_OK ||
        (s = check4(name, "losses", losses, true)) != BQ_OK)
        return s;
    if (bias && scoring != BQ_SCORE_SOFTMAX)
        return bq::fail(BQ_ERR_SHAPE, "%s: under rule %d the bias only selects: pass NULL", name, scoring);
    const size_t need = bq_moe_balance_workspace_bytes(T, E, S);
    if (!workspace || workspace_bytes < need)
        return bq::fail(BQ_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu", name, workspace_bytes, need);
    if (!bq::aligned(workspace, 256)) return bq::fail(BQ_ERR_ALIGN, "%s: workspace must be 256-byte aligned", name);
    if ((s = bq::check_arch()) != BQ_OK) return s;
    const Chunking c = balance_chunking(T);
    const size_t slots = (size_t)c.chunks + S;
    uint8_t* base = static_cast<uint8_t*>(workspace);
    const BalanceArgs a{logits, bias, T, E, k, ids, seq_offsets, S, c.rows, c.chunks, reinterpret_cast<float*>(base),
                        reinterpret_cast<int32_t*>(base + up256(slots * E * 4)),
                        reinterpret_cast<float*>(base + 2 * up256(slots * E * 4)), counts, probs, losses,
                        bq::device_status_ptr()};
    const bool one = T <= kOneClusterRows;
    const int share = share_of((int64_t)slots, S);
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = cudaSuccess;
    with_nper(E, [&](auto nper) {
        constexpr int N = decltype(nper)::value;
        auto go = [&](auto kernel) {
            if ((e = allow_smem(kernel, balance_smem(E))) != cudaSuccess) return;
            if (one) e = launch_cluster(kernel, std::max(1, c.chunks), balance_smem(E), st, a, share);
            else e = bq::launch_after(kernel, dim3(c.chunks), dim3(kThreads), balance_smem(E), st, a, share);
        };
        if (scoring == BQ_SCORE_SQRTSOFTPLUS) one ? go(balance_kernel<N, RULE_SCORE, true>) : go(balance_kernel<N, RULE_SCORE, false>);
        else one ? go(balance_kernel<N, RULE_SOFTMAX, true>) : go(balance_kernel<N, RULE_SOFTMAX, false>);
    });
    if ((s = launched(name, e)) != BQ_OK || one) return s;
    return launched(name, launch_cluster(balance_finish_kernel, 8, 0, st, a, share));
}

extern "C" size_t bq_moe_route_backward_workspace_bytes(int32_t T, int32_t E) {
    if (T < 0 || E < 1 || E > 1024) return 0;
    return up256((size_t)std::max(1, gradient_chunking(T).chunks) * E * 4);
}

extern "C" bq_status bq_moe_route_backward(const float* logits, const float* bias, int32_t T, int32_t E,
                                           const int32_t* ids, int32_t k, int32_t scoring, float scale,
                                           const float* dweights, const int32_t* counts, const float* dlosses,
                                           const int32_t* seq_offsets, int32_t S, void* dlogits, int32_t dtype,
                                           float* dbias, void* workspace, size_t workspace_bytes, bq_stream_t stream) {
    const char* name = "bq_moe_route_backward";
    bq_status s = check_router(name, T, E, k, scoring, seq_offsets, S);
    const int es = bq::dtype_size(dtype);
    if (s == BQ_OK && es == 0) s = bq::fail(BQ_ERR_FORMAT, "%s: unknown element type %d", name, dtype);
    if (s == BQ_OK && T > 0 && !dweights && !dlosses) s = bq::fail(BQ_ERR_NULL, "%s: dweights and dlosses are both NULL", name);
    if (s != BQ_OK || (s = check4(name, "logits", logits, T > 0)) != BQ_OK ||
        (s = check4(name, "bias", bias, false)) != BQ_OK ||
        (s = check4(name, "ids", ids, T > 0 && dweights)) != BQ_OK ||
        (s = check4(name, "dweights", dweights, false)) != BQ_OK ||
        (s = check4(name, "dlosses", dlosses, false)) != BQ_OK ||
        (s = check4(name, "counts", counts, dlosses)) != BQ_OK ||
        (s = check4(name, "seq_offsets", seq_offsets, false)) != BQ_OK ||
        (s = check4(name, "dbias", dbias, false)) != BQ_OK)
        return s;
    if (T > 0 && !dlogits) return bq::fail(BQ_ERR_NULL, "%s: dlogits is NULL", name);
    if (!bq::aligned(dlogits, es)) return bq::fail(BQ_ERR_ALIGN, "%s: dlogits must be aligned to its element", name);
    if ((bias || dbias) && scoring != BQ_SCORE_SOFTMAX)
        return bq::fail(BQ_ERR_SHAPE, "%s: under rule %d the bias only selects: pass NULL, it has no gradient", name, scoring);
    const Chunking c = gradient_chunking(T);
    if (dbias) {
        const size_t need = bq_moe_route_backward_workspace_bytes(T, E);
        if (!workspace || workspace_bytes < need)
            return bq::fail(BQ_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu", name, workspace_bytes, need);
        if (!bq::aligned(workspace, 256)) return bq::fail(BQ_ERR_ALIGN, "%s: workspace must be 256-byte aligned", name);
    }
    if (T == 0 && !dbias) return BQ_OK;
    if ((s = bq::check_arch()) != BQ_OK) return s;
    cudaStream_t st = (cudaStream_t)stream;
    const RouteGradArgs a{logits, bias, T, E, k, ids, dweights, scale, counts, dlosses, seq_offsets, S, c.rows, dlogits,
                          dtype, dbias ? static_cast<float*>(workspace) : nullptr, bq::device_status_ptr()};
    if (T > 0) {
        const size_t smem = dbias ? (size_t)kWarps * E * 4 : 0;
        cudaError_t e = cudaSuccess;
        with_nper(E, [&](auto nper) {
            constexpr int N = decltype(nper)::value;
            auto go = [&](auto kernel) {
                if ((e = allow_smem(kernel, smem)) != cudaSuccess) return;
                e = bq::launch_after(kernel, dim3(c.chunks), dim3(kThreads), smem, st, a);
            };
            if (scoring == BQ_SCORE_SQRTSOFTPLUS)
                dlosses ? go(route_backward_kernel<N, RULE_SCORE, true>) : go(route_backward_kernel<N, RULE_SCORE, false>);
            else
                dlosses ? go(route_backward_kernel<N, RULE_SOFTMAX, true>) : go(route_backward_kernel<N, RULE_SOFTMAX, false>);
        });
        if ((s = launched(name, e)) != BQ_OK) return s;
    }
    if (!dbias) return BQ_OK;
    return launched(name, bq::launch_after(column_sums_kernel, dim3((E + 31) / 32), dim3(kThreads), 0, st,
                                           (const float*)workspace, T > 0 ? c.chunks : 0, E, dbias));
}
