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
//
// A warp takes a row, its logits in registers, the next row's on their way.  The logits are read once (and the
// gradient written once), but issue bounds both passes before memory does (GB300, 16384 x 256, k = 8): the statistics
// of scores over 9 sequences take 13.4 us, 2.5 at the copy bandwidth, of which the first kernel has 8 (three
// special-function instructions a logit, packed arithmetic, 55% of the issue slots at 30 warps an SM; 3.4 rows a warp
// leave a fifth of the last round idle) and the second, a chain of latencies, 5; those of a softmax rule take 10.9.  The
// gradient of weights and losses takes 10.3 us under a softmax rule and 17.8 under the score rule, 5.1 at the copy
// bandwidth, that of the weights alone 7.7.  From 513 experts on a lane holds 32 of them, and the gradient under the score
// rule does not fit its 128 registers (about 500 bytes a thread are spilled): 16384 x 1024 50 us, under a softmax rule 32,
// 19.9 at the copy bandwidth; statistics 29 and 23, at the copy bandwidth 9.9.  Few rows are latency (129 x 128: statistics
// 6.2 us, gradient of weights alone 4.1).
#include <algorithm>
#include <atomic>

#include "packed_f32.cuh"
#include "row_types.cuh"

namespace {

using namespace bq;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSequences = 65536;
constexpr int kMaxExperts = 1024;
constexpr int kMaxRows = INT32_MAX - 64;   // a warp's row behind its last, 16 further on, is still an int
constexpr float kLog2E = 1.4426950408889634f;

enum { RULE_SOFTMAX = 0, RULE_SCORE = 1 };

__device__ __forceinline__ float warp_max(float v) {
    // as ordered integers, one instruction; a NaN that is lost here is met again in the sum of exponentials
    const int i = __float_as_int(v), m = __reduce_max_sync(0xffffffffu, i ^ ((i >> 31) & 0x7fffffff));
    return __int_as_float(m ^ ((m >> 31) & 0x7fffffff));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// exp2, reciprocal and square root of the special-function unit: off by 2 units in the last place at most, results and
// arguments below the normal range become 0.  exp(v) = exp2(v log2 e) is off by |v| units more, from the argument.
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

__device__ __forceinline__ float sqrt_approx(float v) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float log_approx(float v) {   // off by 2^-22 and 2 units in the last place
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r * 0.69314718055994531f;
}

// log(1 + e) / e for e in [0, 1]: a polynomial fitted to it (largest relative error 5e-9, 1.2e-7 evaluated in fp32).
__device__ __forceinline__ f32x2 log1p_ratio(f32x2 e) {
    f32x2 q = fma2(e, both(-0.003243980884f), both(0.01985126273f));
    q = fma2(q, e, both(-0.05695915927f));
    q = fma2(q, e, both(0.1060361689f));
    q = fma2(q, e, both(-0.1530557013f));
    q = fma2(q, e, both(0.1967593147f));
    q = fma2(q, e, both(-0.2495413214f));
    q = fma2(q, e, both(0.3332996227f));
    q = fma2(q, e, both(-0.4999990242f));
    return fma2(q, e, both(0.9999999953f));
}

// sqrt(softplus(z)) of two logits.  With h = exp(-|z| / 2) and e = h^2, softplus is max(z, 0) + log(1 + e); below 0 its
// root is h sqrt(log(1 + e) / e), which loses nothing where e does (h is normal down to z = -174).  slope: with the
// derivative sigmoid(z) / (2 score) too.
template <bool SLOPE>
__device__ __forceinline__ void scores_of(float z0, float z1, float& s0, float& s1, float& d0, float& d1) {
    const float2 a = parts_of(mul2(two(fabsf(z0), fabsf(z1)), both(-0.5f * kLog2E)));
    const f32x2 h = two(exp2_approx(a.x), exp2_approx(a.y)), e = mul2(h, h), ratio = log1p_ratio(e);
    const float2 hs = parts_of(h), low = parts_of(ratio), soft = parts_of(fma2(e, ratio, two(fmaxf(z0, 0.f), fmaxf(z1, 0.f))));
    const float r0 = sqrt_approx(z0 < 0.f ? low.x : soft.x), r1 = sqrt_approx(z1 < 0.f ? low.y : soft.y);
    s0 = z0 < 0.f ? hs.x * r0 : r0;
    s1 = z1 < 0.f ? hs.y * r1 : r1;
    if (SLOPE) {   // sigmoid(z) is 1 / (1 + e) from 0 on and e / (1 + e) below
        const float2 den = parts_of(mul2(fma2(e, both(2.f), both(2.f)), two(r0, r1)));
        d0 = (z0 < 0.f ? hs.x : 1.f) * rcp_approx(den.x);
        d1 = (z1 < 0.f ? hs.y : 1.f) * rcp_approx(den.y);
    }
}

// A warp's share of a row: lane l holds experts at(l, i), i < NPER: four in a row at a time where rows lie on 16-byte
// boundaries (VEC), else 32 apart.  Values behind the last expert are -inf.
template <int NPER, bool VEC>
struct Share {
    static __device__ __forceinline__ int at(int lane, int i) { return VEC ? 128 * (i >> 2) + 4 * lane + (i & 3) : lane + 32 * i; }

    static __device__ __forceinline__ void load(const float* row, const float* bias, int E, int lane, float (&z)[NPER]) {
        if (VEC) {
#pragma unroll
            for (int i = 0; i < NPER; i += 4) {
                const bool in = at(lane, i) < E;
                const float4 v = in ? __ldg(reinterpret_cast<const float4*>(row + at(lane, i)))
                                    : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                z[i] = v.x; z[(i + 1) % NPER] = v.y; z[(i + 2) % NPER] = v.z; z[(i + 3) % NPER] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < NPER; ++i) z[i] = at(lane, i) < E ? __ldg(row + at(lane, i)) : -INFINITY;
        }
        if (bias) {
#pragma unroll
            for (int i = 0; i < NPER; ++i)
                if (at(lane, i) < E) z[i] = __fadd_rn(z[i], __ldg(bias + at(lane, i)));
        }
    }

    static __device__ __forceinline__ void store(void* matrix, int64_t row, int dtype, int E, int lane, const float (&v)[NPER]) {
        if (VEC) {
#pragma unroll
            for (int i = 0; i < NPER; i += 4) {
                if (at(lane, i) >= E) continue;
                const int64_t to = row * E + at(lane, i);
                const float f[4] = {v[i], v[(i + 1) % NPER], v[(i + 2) % NPER], v[(i + 3) % NPER]};
                if (dtype == BQ_DT_F32) {
                    *reinterpret_cast<float4*>(static_cast<float*>(matrix) + to) = make_float4(f[0], f[1], f[2], f[3]);
                } else if (dtype == BQ_DT_F16) {
                    *reinterpret_cast<uint2*>(static_cast<__half*>(matrix) + to) =
                        make_uint2(h2_as_u32(__floats2half2_rn(f[0], f[1])), h2_as_u32(__floats2half2_rn(f[2], f[3])));
                } else {
                    const __nv_bfloat162 lo = __floats2bfloat162_rn(f[0], f[1]), hi = __floats2bfloat162_rn(f[2], f[3]);
                    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(matrix) + to) =
                        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < NPER; ++i)
                if (at(lane, i) < E) store_value(matrix, row * E + at(lane, i), dtype, v[i]);
        }
    }
};

// What the softmax of a row is made of: its largest logit m (0 for a row of -inf only), 1 / the sum of exp(z - m) and
// the log-sum-exp (both 0 for such a row).
struct Softmax {
    float m, inv, lse;
};

// ex: the exponentials.
template <int NPER>
__device__ __forceinline__ Softmax softmax_row(const float (&z)[NPER], float (&ex)[NPER]) {
    float m = z[0];
#pragma unroll
    for (int i = 1; i < NPER; ++i) m = fmaxf(m, z[i]);
    m = warp_max(m);
    if (m == -INFINITY) m = 0.f;
    float sum = 0.f;
    if (NPER == 1) {
        sum = ex[0] = exp2_approx((z[0] - m) * kLog2E);
    } else {
        f32x2 total = both(0.f);
#pragma unroll
        for (int i = 0; i < NPER; i += 2) {
            const int j = (i + 1) % NPER;
            const float2 d = parts_of(mul2(fma2(two(z[i], z[j]), both(1.f), both(-m)), both(kLog2E)));
            ex[i] = exp2_approx(d.x);
            ex[j] = exp2_approx(d.y);
            total = fma2(two(ex[i], ex[j]), both(1.f), total);
        }
        sum = sum2(total);
    }
    sum = warp_sum(sum);
    return {m, sum == 0.f ? 0.f : rcp_approx(sum), sum == 0.f ? 0.f : m + log_approx(sum)};
}

// <x, y> over the warp's row.
template <int NPER>
__device__ __forceinline__ float row_dot(const float (&x)[NPER], const float (&y)[NPER]) {
    if (NPER == 1) return warp_sum(x[0] * y[0]);
    f32x2 dot = both(0.f);
#pragma unroll
    for (int i = 0; i < NPER; i += 2) dot = fma2(two(x[i], x[(i + 1) % NPER]), two(y[i], y[(i + 1) % NPER]), dot);
    return warp_sum(sum2(dot));
}

// Where a row's largest logit m lies below this, e = exp(z) is less than 2^-28, and a score is exp(z / 2) to fp32's
// precision.  exp(m / 2) cancels in score / sum and in slope / sum, and is left out of both: far below 0 (z < -174) the
// scores themselves are below fp32's normal range.
constexpr float kFarBelow = -20.f;

__device__ __forceinline__ float far_score(float z, float m) { return exp2_approx((z - m) * (0.5f * kLog2E)); }

// Scores (and slopes) of a row, and 1 / their sum (0 where every score is 0); both without the factor exp(m / 2) where the
// largest logit m (0 for a row of -inf only) is below kFarBelow.
template <bool SLOPE, int NPER>
__device__ __forceinline__ float score_row(const float (&z)[NPER], float m, float (&s)[NPER], float (&d)[NPER]) {
    float sum = 0.f;
    if (m < kFarBelow) {
#pragma unroll
        for (int i = 0; i < NPER; ++i) {
            s[i] = far_score(z[i], m);
            if (SLOPE) d[i] = 0.5f * s[i];
            sum += s[i];
        }
    } else if (NPER == 1) {
        float unused0, unused1;
        scores_of<SLOPE>(z[0], 0.f, s[0], unused0, d[0], unused1);
        sum = s[0];
    } else {
#pragma unroll
        for (int i = 0; i < NPER; i += 2) {
            scores_of<SLOPE>(z[i], z[(i + 1) % NPER], s[i], s[(i + 1) % NPER], d[i], d[(i + 1) % NPER]);
            sum += s[i] + s[(i + 1) % NPER];
        }
    }
    sum = warp_sum(sum);   // what lies behind the last expert has z = -inf and adds 0
    return sum == 0.f ? 0.f : rcp_approx(sum);
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

struct Totals {
    int used, rows;   // sequences that have rows, and their rows
    int before;       // sequences that end at `row` or before it: the first that does not
};

// All threads of the CTA; contains barriers.
__device__ __forceinline__ Totals sequence_totals(const int32_t* offsets, int S, int T, int row, int32_t* status) {
    __shared__ int s_totals[3];
    if (!offsets) return {T > 0, T, 0};
    if (threadIdx.x < 3) s_totals[threadIdx.x] = 0;
    __syncthreads();
    int used = 0, rows = 0, before = 0;
    for (int s = threadIdx.x; s < S; s += blockDim.x) {
        int lo, hi;
        before += __ldg(offsets + s + 1) <= row;
        if (sequence(offsets, s, T, status, lo, hi) && hi > lo) { ++used; rows += hi - lo; }
    }
    if (used | before) {
        atomicAdd(&s_totals[0], used);
        atomicAdd(&s_totals[1], rows);
        atomicAdd(&s_totals[2], before);
    }
    __syncthreads();
    return {s_totals[0], s_totals[1], s_totals[2]};
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
    float* part_loss;    // [S * groups of 32 experts][2]
    int* ended;          // CTAs of balance_finish_kernel that have ended; sequences that have rows; their rows
    int32_t* counts;
    float* probs;
    float* losses;
    int32_t* status;
};

// The rows are cut into chunks of equal size, a CTA each, whatever sequences they belong to: one long sequence among
// short ones takes no longer than many of equal length.  Chunk c leaves its sums over sequence s in slot c + s: along
// rows that ascend, either c or s grows from one (chunk, sequence) to the next, so no two share a slot.
template <int NPER, bool VEC, int RULE>
__device__ __forceinline__ void chunk_sums(const BalanceArgs& a, float* s_red, int32_t* s_hist) {
    using Row = Share<NPER, VEC>;
    constexpr bool kAhead = NPER <= 8;   // the next row is loaded ahead, where there are registers for it
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t first = (int64_t)blockIdx.x * a.chunk_rows;
    const int row0 = (int)first, row1 = (int)min((int64_t)a.T, first + a.chunk_rows);
    float z[NPER];
    if (kAhead && row0 + warp < row1) Row::load(a.logits + (int64_t)(row0 + warp) * a.E, a.bias, a.E, lane, z);
    const Totals totals = sequence_totals(a.offsets, a.S, a.T, row0, a.status);
    if (blockIdx.x == 0 && threadIdx.x == 0) {   // for balance_finish_kernel
        a.ended[0] = 0;
        a.ended[1] = totals.used;
        a.ended[2] = totals.rows;
    }
    for (int s = totals.before; s < a.S; ++s) {
        int lo, hi;
        sequence(a.offsets, s, a.T, a.status, lo, hi);
        if (lo >= row1) break;
        lo = max(lo, row0);
        hi = min(hi, row1);
        if (lo >= hi) continue;
        for (int e = threadIdx.x; e < a.E; e += kThreads) s_hist[e] = 0;
        float acc[NPER], z2 = 0.f;
        if (kAhead && lo > row0 && lo + warp < hi) Row::load(a.logits + (int64_t)(lo + warp) * a.E, a.bias, a.E, lane, z);
        __syncthreads();
        for (int64_t i = (int64_t)lo * a.k + threadIdx.x; i < (int64_t)hi * a.k; i += kThreads) {
            const int e = __ldg(a.ids + i);
            if (e >= 0 && e < a.E) atomicAdd(&s_hist[e], 1);
            else bq::set_device_error(a.status, BQ_DEV_BAD_EXPERT_ID);
        }
#pragma unroll
        for (int i = 0; i < NPER; ++i) acc[i] = 0.f;
        for (int r = lo + warp; r < hi; r += kWarps) {
            float next[NPER], p[NPER], unused[NPER];
            if (!kAhead) Row::load(a.logits + (int64_t)r * a.E, a.bias, a.E, lane, z);
            else if (r + kWarps < hi) Row::load(a.logits + (int64_t)(r + kWarps) * a.E, a.bias, a.E, lane, next);
            const Softmax soft = softmax_row(z, p);
            float inv = soft.inv;
            if (RULE == RULE_SCORE) inv = score_row<false>(z, soft.m, p, unused);
#pragma unroll
            for (int i = 0; i < NPER; ++i) {
                acc[i] = __fmaf_rn(p[i], inv, acc[i]);
                if (kAhead) z[i] = next[i];
            }
            z2 = __fmaf_rn(soft.lse, soft.lse, z2);
        }
#pragma unroll
        for (int i = 0; i < NPER; ++i)
            if (Row::at(lane, i) < a.E) s_red[warp * a.E + Row::at(lane, i)] = acc[i];
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

// One warp's share of the slots of a group, 32 experts of a sequence (rows [lo, hi)): slots sub, sub + share, ...
struct GroupSums {
    float p;
    int c;
    float z2;    // per lane, of the first group of a sequence
};

__device__ __forceinline__ GroupSums add_slots(const BalanceArgs& a, int s, int block, int lo, int hi, int sub, int share) {
    const int lane = threadIdx.x & 31, e = block * 32 + lane;
    GroupSums r{0.f, 0, 0.f};
    if (hi <= lo) return r;
    const int64_t begin = lo / a.chunk_rows + (int64_t)s, end = (hi - 1) / a.chunk_rows + (int64_t)s + 1;
    if (e < a.E) {
        const float* from_p = a.part_p + e;
        const int32_t* from_c = a.part_c + e;
        int64_t i = begin + sub;
        for (; i + 7 * share < end; i += 8 * share) {   // eight slots in flight together
            float p[8];
            int c[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                p[j] = from_p[(i + j * share) * a.E];
                c[j] = from_c[(i + j * share) * a.E];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                r.p += p[j];
                r.c += c[j];
            }
        }
#pragma unroll 4
        for (; i < end; i += share) {
            r.p += from_p[i * a.E];
            r.c += from_c[i * a.E];
        }
    }
    if (block == 0)
        for (int64_t i = begin + 32 * sub + lane; i < end; i += 32 * share) r.z2 += a.part_z[i];
    return r;
}

// Counts and mean probability of an expert; its share of the balance loss.
__device__ __forceinline__ float write_group(const BalanceArgs& a, int s, int e, int lo, int hi, float p, int c) {
    const float n = (float)(hi - lo), mean = hi > lo ? p / n : 0.f;
    a.counts[(int64_t)s * a.E + e] = c;
    a.probs[(int64_t)s * a.E + e] = mean;
    return hi > lo ? (float)c * ((float)a.E / ((float)a.k * n)) * mean : 0.f;
}

// The slots of every sequence added up, by the CTAs of one cluster; `share` warps (a power of two) have a share of a
// group's slots each.  s_red, s_redc: a word per thread.
__device__ __forceinline__ void finish(const BalanceArgs& a, int rank, int ranks, int share, float* s_red, int32_t* s_redc) {
    __shared__ float s_loss[2][kWarps];
    __shared__ float s_cta[2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Totals totals = sequence_totals(a.offsets, a.S, a.T, 0, a.status);
    const int blocks = (a.E + 31) / 32, sub = warp & (share - 1), at_once = kWarps / share;
    const int64_t groups = (int64_t)a.S * blocks;
    float balance = 0.f, z2 = 0.f;
    for (int64_t g0 = (int64_t)rank * at_once; g0 < groups; g0 += (int64_t)ranks * at_once) {
        const int64_t g = g0 + warp / share;
        const int s = (int)(g / blocks), block = (int)(g - (int64_t)s * blocks), e = block * 32 + lane;
        int lo = 0, hi = 0;
        if (g < groups) sequence(a.offsets, s, a.T, a.status, lo, hi);
        GroupSums r = add_slots(a, s, block, lo, hi, sub, share);
        z2 += r.z2;
        if (share > 1) {
            s_red[threadIdx.x] = r.p;
            s_redc[threadIdx.x] = r.c;
            __syncthreads();
            if (sub == 0) {
                for (int w = 1; w < share; ++w) {
                    r.p += s_red[threadIdx.x + 32 * w];
                    r.c += s_redc[threadIdx.x + 32 * w];
                }
            }
            __syncthreads();
        }
        if (sub == 0 && g < groups && e < a.E) balance += write_group(a, s, e, lo, hi, r.p, r.c);
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
        const int n = threadIdx.x ? totals.rows : totals.used;
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

// one: the launch is one cluster, which also adds its slots up.
template <int NPER, bool VEC, int RULE>
__global__ void __launch_bounds__(kThreads, NPER <= 8 ? 2 : 1)
balance_kernel(const __grid_constant__ BalanceArgs a, int share, int one) {
    extern __shared__ float s_dyn[];
    bq::grid_dependency_wait();   // launched behind whatever precedes it on the stream
    bq::allow_dependents();
    int32_t* hist = reinterpret_cast<int32_t*>(s_dyn + sums_words(a.E));
    chunk_sums<NPER, VEC, RULE>(a, s_dyn, hist);
    if (one) {
        const int ranks = gridDim.x;
        if (ranks > 1) cluster_sync();   // the slots that the others wrote
        else __syncthreads();
        finish(a, ranks > 1 ? cluster_rank() : 0, ranks, share, s_dyn, hist);
    }
}

// Of many chunks: a CTA per group, its warps a share of the group's slots each (one cluster of 8 CTAs for all groups
// took 25 us in all instead of 14).  The last CTA to end adds the groups'
// losses up, in their order; balance_kernel has set the count of those that ended to 0.
__global__ void __launch_bounds__(kThreads)
balance_finish_kernel(const __grid_constant__ BalanceArgs a) {
    __shared__ float s_red[kWarps][32];
    __shared__ int32_t s_redc[kWarps][32];
    __shared__ float s_sum[2][kWarps];
    __shared__ int s_last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, blocks = (a.E + 31) / 32;
    const int s = blockIdx.x / blocks, block = blockIdx.x - s * blocks, e = block * 32 + lane;
    bq::grid_dependency_wait();   // nothing before this line touches global memory, which earlier kernels may have written
    bq::allow_dependents();
    int lo, hi;
    sequence(a.offsets, s, a.T, a.status, lo, hi);
    GroupSums r = add_slots(a, s, block, lo, hi, warp, kWarps);
    s_red[warp][lane] = r.p;
    s_redc[warp][lane] = r.c;
    r.z2 = warp_sum(r.z2);
    if (lane == 0) s_sum[1][warp] = r.z2;
    __syncthreads();
    if (warp == 0) {
        float z2 = 0.f, balance = 0.f;
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            r.p += s_red[w][lane];
            r.c += s_redc[w][lane];
        }
        for (int w = 0; w < kWarps; ++w) z2 += s_sum[1][w];
        if (e < a.E) balance = write_group(a, s, e, lo, hi, r.p, r.c);
        balance = warp_sum(balance);
        if (lane == 0) {
            a.part_loss[2 * blockIdx.x] = balance;
            a.part_loss[2 * blockIdx.x + 1] = z2;
            __threadfence();
            s_last = atomicAdd(a.ended, 1) == (int)gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    const int n = threadIdx.x < 2 ? __ldcg(a.ended + 1 + threadIdx.x) : 0;
    float sum[2] = {0.f, 0.f};
    for (int g = threadIdx.x; g < (int)gridDim.x; g += kThreads) {
        sum[0] += __ldcg(a.part_loss + 2 * g);
        sum[1] += __ldcg(a.part_loss + 2 * g + 1);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        sum[i] = warp_sum(sum[i]);
        if (lane == 0) s_sum[i][warp] = sum[i];
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        float v = 0.f;
        for (int w = 0; w < kWarps; ++w) v += s_sum[threadIdx.x][w];
        a.losses[threadIdx.x] = n ? v / (float)n : 0.f;
    }
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
    float* part_b;           // [chunks][E] sums of the bias gradient, or NULL: it is not wanted
    float* dbias;            // not NULL: the launch is one cluster, and writes it
    int32_t* status;
};

// The selected experts of four of a warp's rows at a time: lane 8 q + j has expert j < k of the q-th (rows lie kWarps
// apart).  One row at a time, k lanes at work, the gradient took 13.3 us instead of 10.3.  Loaded ahead: the id and the
// gradient a batch of four ahead, the logit (a chain of two loads) with them.
struct Pair {
    int id = -1;
    float dw = 0.f, z = -INFINITY;

    __device__ __forceinline__ void load(const RouteGradArgs& a, int64_t first, int row1, int lane) {
        const int64_t r = first + (lane >> 3) * kWarps;
        id = -1;
        if (r >= row1 || (lane & 7) >= a.k) return;
        id = __ldg(a.ids + r * a.k + (lane & 7));
        dw = __ldg(a.dweights + r * a.k + (lane & 7));
    }
    __device__ __forceinline__ void load_logit(const RouteGradArgs& a, int64_t first, int lane) {
        if (id < 0 || id >= a.E) return;
        z = __ldg(a.logits + (first + (lane >> 3) * kWarps) * a.E + id);
        if (a.bias) z = __fadd_rn(z, __ldg(a.bias + id));
    }
    // An id that names no expert, reported when its row's turn comes (if that belongs to a sequence).
    __device__ __forceinline__ void report(const RouteGradArgs& a, int q, int lane) const {
        if (lane >> 3 == q && (lane & 7) < a.k && (id < 0 || id >= a.E)) bq::set_device_error(a.status, BQ_DEV_BAD_EXPERT_ID);
    }
};

__device__ __forceinline__ float sum_of_eight(float v) {
#pragma unroll
    for (int off = 4; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// The gradient that the router weights bring to the four rows: each lane its expert id (-1: none) and its share g.  Of
// lanes that name the same expert of a row the first gets the sum, the others -1.
template <int RULE>
__device__ __forceinline__ void selected(const RouteGradArgs& a, const Pair& p, int lane, int& id, float& g) {
    id = p.id < a.E ? p.id : -1;
    if (id < 0) id = -1;
    if (RULE == RULE_SOFTMAX) {
        float m = id >= 0 ? p.z : -INFINITY;
#pragma unroll
        for (int off = 4; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        if (m == -INFINITY) m = 0.f;   // none selected, or all of them -inf: no weights, no gradient
        const float ex = id >= 0 ? exp2_approx((p.z - m) * kLog2E) : 0.f, total = sum_of_eight(ex);
        const float w = total == 0.f ? 0.f : __fdividef(ex, total), mean = sum_of_eight(id >= 0 ? w * p.dw : 0.f);
        g = id >= 0 ? w * (p.dw - mean) : 0.f;
    } else {
        float score, slope, unused0, unused1;
        scores_of<true>(p.z, 0.f, score, unused0, slope, unused1);
        g = id >= 0 ? a.scale * p.dw * slope : 0.f;
    }
    // the same index twice (a router names none twice, a caller may): added in slot order
    const uint32_t same = __match_any_sync(0xffffffffu, id >= 0 ? 4 * id + (lane >> 3) : ~lane);
    if (__any_sync(0xffffffffu, __popc(same) > 1)) {
        float sum = 0.f;
        for (int j = 0; j < a.k; ++j) {
            const int from = (lane & 24) + j;
            const float gj = __shfl_sync(0xffffffffu, g, from);
            if (same >> from & 1) sum += gj;
        }
        if (__popc(same) > 1) {
            g = sum;
            if (__ffs(same) - 1 != lane) id = -1;
        }
    }
}

// The rows of a CTA's chunk, a warp each, with the sequence that a row belongs to (rows ascend, so sequences do).
struct Place {
    int s, lo, hi;
    bool fresh;   // the sequence changed

    __device__ __forceinline__ bool find(const RouteGradArgs& a, int r) {
        if (!a.offsets) return true;
        while (s < a.S && r >= hi) {
            sequence(a.offsets, s, a.T, a.status, lo, hi);
            fresh = true;
            if (r >= hi) ++s;
        }
        return r >= lo && r < hi;   // rows in none are left out
    }
};

// A chunk's column sums: the warps' sums in warp order.  Where the launch is one cluster, its CTAs add the chunks up at
// once, each a share of the columns, in the order of the chunks.
__device__ __forceinline__ void write_part(const RouteGradArgs& a, float* s_acc) {
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += s_acc[w * a.E + e];
        if (a.dbias) s_acc[e] = sum;   // of the column's own thread, which has read it
        else a.part_b[(int64_t)blockIdx.x * a.E + e] = sum;
    }
    if (!a.dbias) return;
    const int ranks = gridDim.x;
    if (ranks > 1) cluster_sync();
    else __syncthreads();
    for (int e = blockIdx.x * kThreads + threadIdx.x; e < a.E; e += ranks * kThreads) {
        float sum = 0.f;
        for (int r = 0; r < ranks; ++r) sum += ranks > 1 ? peer_load(s_acc + e, r) : s_acc[e];
        a.dbias[e] = sum;
    }
    if (ranks > 1) cluster_sync();   // peers may still be reading
}

// With losses: a warp per row, the row's gradient of the losses in its registers.  Logits are read once and gradients
// written once; the k selected values are then written again by the lanes that hold their share, each from its own
// evaluation of the loss's gradient (cheaper than bringing the shares to the lanes that hold the experts).
template <int NPER, bool VEC, int RULE>
__global__ void __launch_bounds__(kThreads, NPER <= (RULE == RULE_SCORE ? 4 : 8) ? 2 : 1)
route_backward_kernel(const __grid_constant__ RouteGradArgs a) {
    using Row = Share<NPER, VEC>;
    constexpr bool kAhead = NPER <= 8;   // the next row is loaded ahead, where there are registers for it
    extern __shared__ float s_dyn[];   // with part_b: a row of sums per warp
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    bq::grid_dependency_wait();   // launched behind whatever precedes it on the stream
    bq::allow_dependents();
    const int64_t first = (int64_t)blockIdx.x * a.chunk_rows;
    const int row0 = (int)first, row1 = (int)min((int64_t)a.T, first + a.chunk_rows);
    float* s_acc = s_dyn + warp * a.E;
    if (a.part_b)
        for (int e = lane; e < a.E; e += 32) s_acc[e] = 0.f;
    __syncwarp();
    float z[NPER];
    if (kAhead && row0 + warp < row1) Row::load(a.logits + (int64_t)(row0 + warp) * a.E, a.bias, a.E, lane, z);
    Pair pair, ahead;
    if (a.dweights) pair.load(a, (int64_t)row0 + warp, row1, lane);
    const float dbalance = __ldg(a.dlosses), dz = __ldg(a.dlosses + 1);
    const Totals totals = sequence_totals(a.offsets, a.S, a.T, row0, a.status);
    const float per_seq = dbalance * ((float)a.E / (float)a.k) / (float)max(1, totals.used);
    const float per_row = 2.f * dz / (float)max(1, totals.rows);
    if (a.dweights) pair.load_logit(a, (int64_t)row0 + warp, lane);
    Place place{totals.before, a.offsets ? -1 : 0, a.offsets ? -1 : a.T, true};
    float acc[NPER], weight[NPER], per_count = 0.f;
#pragma unroll
    for (int i = 0; i < NPER; ++i) acc[i] = weight[i] = 0.f;
    int id = -1, q = 0;
    float g = 0.f;
    for (int r = row0 + warp; r < row1; r += kWarps) {
        float next[NPER];
        if (!kAhead) Row::load(a.logits + (int64_t)r * a.E, a.bias, a.E, lane, z);
        else if (r + kWarps < row1) Row::load(a.logits + (int64_t)(r + kWarps) * a.E, a.bias, a.E, lane, next);
        if (a.dweights) {
            if (q == 0) {
                selected<RULE>(a, pair, lane, id, g);
                ahead.load(a, (int64_t)r + 4 * kWarps, row1, lane);
            } else if (q == 1) {
                ahead.load_logit(a, (int64_t)r + 3 * kWarps, lane);
            }
        }
        if (place.find(a, r)) {
            const int32_t* counts = a.counts + (int64_t)place.s * a.E;
            if (place.fresh) {
                const float n = (float)(place.hi - place.lo);
                per_count = per_seq / n / n;
#pragma unroll
                for (int i = 0; i < NPER; ++i)
                    weight[i] = Row::at(lane, i) < a.E ? (float)__ldg(counts + Row::at(lane, i)) * per_count : 0.f;
                place.fresh = false;
            }
            const bool mine = lane >> 3 == q && id >= 0;
            const float own = mine ? (float)__ldg(counts + id) * per_count : 0.f;
            float d[NPER], base = 0.f;
            const Softmax soft = softmax_row(z, d);
            const float f = per_row * soft.lse * soft.inv;
            if (RULE == RULE_SOFTMAX) {
                // p (weight - <p, weight> + per_row lse), p = d inv
                const float rest = __fmaf_rn(-row_dot(d, weight) * soft.inv, soft.inv, f);
#pragma unroll
                for (int i = 0; i < NPER; ++i) d[i] *= __fmaf_rn(weight[i], soft.inv, rest);
                if (mine) base = exp2_approx((pair.z - soft.m) * kLog2E) * __fmaf_rn(own, soft.inv, rest);
            } else {
                float sc[NPER], slope[NPER];
                const float inv = score_row<true>(z, soft.m, sc, slope), dot = row_dot(sc, weight) * inv;
#pragma unroll
                for (int i = 0; i < NPER; ++i) d[i] = __fmaf_rn(d[i], f, slope[i] * inv * (weight[i] - dot));
                if (mine) {
                    float score, change, unused0, unused1;
                    if (soft.m < kFarBelow) change = 0.5f * far_score(pair.z, soft.m);
                    else scores_of<true>(pair.z, 0.f, score, unused0, change, unused1);
                    base = __fmaf_rn(exp2_approx((pair.z - soft.m) * kLog2E), f, change * inv * (own - dot));
                }
            }
            Row::store(a.dlogits, r, a.dtype, a.E, lane, d);
            __syncwarp();   // the row is written before its selected values are written again
            if (mine) store_value(a.dlogits, (int64_t)r * a.E + id, a.dtype, base + g);
            if (a.dweights) pair.report(a, q, lane);
            if (a.part_b) {
                if (mine) s_acc[id] += g;
                __syncwarp();
#pragma unroll
                for (int i = 0; i < NPER; ++i) acc[i] += d[i];
            }
        }
        if (++q == 4) {
            q = 0;
            pair = ahead;
        }
        if (kAhead) {
#pragma unroll
            for (int i = 0; i < NPER; ++i) z[i] = next[i];
        }
    }
    if (!a.part_b) return;
#pragma unroll
    for (int i = 0; i < NPER; ++i)
        if (Row::at(lane, i) < a.E) s_acc[Row::at(lane, i)] += acc[i];
    write_part(a, s_dyn);
}

// Without losses: only the k selected values differ from 0, and only their logits are read.  wide: rows of 16-byte
// vectors.
template <int RULE>
__global__ void __launch_bounds__(kThreads)
route_weights_backward_kernel(const __grid_constant__ RouteGradArgs a, int wide) {
    extern __shared__ float s_dyn[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    bq::grid_dependency_wait();   // launched behind whatever precedes it on the stream
    bq::allow_dependents();
    const int64_t first = (int64_t)blockIdx.x * a.chunk_rows;
    const int row0 = (int)first, row1 = (int)min((int64_t)a.T, first + a.chunk_rows);
    const int es = a.dtype == BQ_DT_F32 ? 4 : 2;
    float* s_acc = s_dyn + warp * a.E;
    if (a.part_b)
        for (int e = lane; e < a.E; e += 32) s_acc[e] = 0.f;
    __syncwarp();
    Place place{sequence_totals(a.offsets, a.S, a.T, row0, a.status).before, a.offsets ? -1 : 0, a.offsets ? -1 : a.T, true};
    Pair pair;
    int id = -1, q = 0;
    float g = 0.f;
    for (int r = row0 + warp; r < row1; r += kWarps, q = (q + 1) & 3) {
        if (q == 0) {
            pair.load(a, r, row1, lane);
            pair.load_logit(a, r, lane);
            selected<RULE>(a, pair, lane, id, g);
        }
        if (!place.find(a, r)) continue;
        uint8_t* row = static_cast<uint8_t*>(a.dlogits) + (int64_t)r * a.E * es;
        if (wide) {
            for (int i = lane; i < a.E * es / 16; i += 32) reinterpret_cast<uint4*>(row)[i] = make_uint4(0, 0, 0, 0);
        } else {
            for (int i = lane; i < a.E; i += 32) store_value(row, i, a.dtype, 0.f);
        }
        __syncwarp();   // the zeros are written before the values
        if (lane >> 3 == q && id >= 0) {
            store_value(row, id, a.dtype, g);
            if (a.part_b) s_acc[id] += g;
        }
        pair.report(a, q, lane);
        __syncwarp();
    }
    if (a.part_b) write_part(a, s_dyn);
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

// As many rows go to one cluster, which adds its chunks' sums up itself: what a second launch costs the host (1.2 us) is
// saved, and on the GPU both take the same (200 x 256: statistics 6.1 us, gradient with that of the bias 5.8 and 5.6 in
// two launches; 400 x 128 6.5 and 6.0, 6.4 and 4.8).  With more than a few sequences the one cluster takes longer than a
// block per group would (17 and 64 sequences: 200 x 256 11.2 and 20.1 us, in two launches 9.5 and 16.3; 200 x 1024 18.6
// and 40.8, 15.5 and 30.3; 16 x 1024, one block, 47.6 and 114, 27.1 and 50.3).
constexpr int kOneClusterRows = 256;

Chunking balance_chunking(int T) { return T <= kOneClusterRows ? chunking(T, 8, kWarps) : chunking(T, 2 * kSms, kWarps); }

// There the cluster is for the sums of a bias gradient.
Chunking gradient_chunking(int T, bool bias) {
    return bias && T <= kOneClusterRows ? chunking(T, 8, kWarps) : chunking(T, 2 * kSms, kWarps);
}

// Calls f with the experts of a lane and whether they are taken four at a time.
template <typename F>
void with_share(int E, bool vec, F f) {
    const std::true_type yes;
    const std::false_type no;
    if (E <= 32) f(std::integral_constant<int, 1>(), no);
    else if (E <= 64) f(std::integral_constant<int, 2>(), no);
    else if (E <= 128) vec ? f(std::integral_constant<int, 4>(), yes) : f(std::integral_constant<int, 4>(), no);
    else if (E <= 256) vec ? f(std::integral_constant<int, 8>(), yes) : f(std::integral_constant<int, 8>(), no);
    else if (E <= 512) vec ? f(std::integral_constant<int, 16>(), yes) : f(std::integral_constant<int, 16>(), no);
    else vec ? f(std::integral_constant<int, 32>(), yes) : f(std::integral_constant<int, 32>(), no);
}

bq_status check_router(const char* name, int T, int E, int k, int scoring, const int32_t* offsets, int S) {
    if (T < 0 || T > kMaxRows) return bq::fail(BQ_ERR_SHAPE, "%s: T = %d outside [0, %d]", name, T, kMaxRows);
    if (E < 1 || E > kMaxExperts) return bq::fail(BQ_ERR_SHAPE, "%s: E = %d outside [1, %d]", name, E, kMaxExperts);
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

// Lets a kernel take more shared memory than 48 KB: the most that any call needs, set once per device (the attribute is a
// property of the function on the current device; set to each call's own size, it could be lowered by another host thread
// before a launch that needs more).
template <auto kernel>
cudaError_t allow_smem(size_t smem) {
    if (smem <= 48 * 1024) return cudaSuccess;
    static std::atomic<bool> attr_set[64];
    int dev = 0;
    cudaGetDevice(&dev);
    const bool known = dev >= 0 && dev < 64;
    if (known && attr_set[dev].load(std::memory_order_acquire)) return cudaSuccess;
    const size_t most = balance_smem(kMaxExperts);
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e == cudaSuccess && known) attr_set[dev].store(true, std::memory_order_release);
    return e;
}

template <auto kernel>
using Constant = std::integral_constant<decltype(kernel), kernel>;   // a kernel as an argument

// Warps that share a group of 32 experts of a sequence: as many as there are for it, but two slots each at least.
int share_of(int warps, int64_t slots, int S, int E) {
    const int64_t groups = (int64_t)S * ((E + 31) / 32);
    int share = 1;
    while (share < kWarps && 2 * share * groups <= warps && slots / S >= 4 * share) share *= 2;
    return share;
}

}  // namespace

extern "C" size_t bq_moe_balance_workspace_bytes(int32_t T, int32_t E, int32_t S) {
    if (T < 0 || T > kMaxRows || E < 1 || E > kMaxExperts || S < 1 || S > kMaxSequences) return 0;
    const size_t slots = (size_t)balance_chunking(T).chunks + S;
    return 2 * up256(slots * E * 4) + up256(slots * 4) + up256((size_t)S * ((E + 31) / 32) * 8) + 256;
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
                        reinterpret_cast<float*>(base + 2 * up256(slots * E * 4)),
                        reinterpret_cast<float*>(base + 2 * up256(slots * E * 4) + up256(slots * 4)),
                        reinterpret_cast<int*>(base + need - 256), counts, probs, losses, bq::device_status_ptr()};
    const bool one = T <= kOneClusterRows, vec = E % 4 == 0 && bq::aligned(logits, 16);
    const int ctas = std::max(1, c.chunks);
    const int share = share_of(ctas * kWarps, slots, S, E);
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = cudaSuccess;
    with_share(E, vec, [&](auto nper, auto v) {
        constexpr int N = decltype(nper)::value;
        constexpr bool VEC = decltype(v)::value;
        auto go = [&](auto constant) {
            constexpr auto kernel = decltype(constant)::value;
            if ((e = allow_smem<kernel>(balance_smem(E))) != cudaSuccess) return;
            if (one) e = launch_cluster(kernel, ctas, balance_smem(E), st, a, share, 1);
            else e = bq::launch_after(kernel, dim3(ctas), dim3(kThreads), balance_smem(E), st, a, share, 0);
        };
        if (scoring == BQ_SCORE_SQRTSOFTPLUS) go(Constant<balance_kernel<N, VEC, RULE_SCORE>>());
        else go(Constant<balance_kernel<N, VEC, RULE_SOFTMAX>>());
    });
    if ((s = launched(name, e)) != BQ_OK || one) return s;
    return launched(name, bq::launch_after(balance_finish_kernel, dim3((unsigned)(S * ((E + 31) / 32))), dim3(kThreads), 0,
                                           st, a));
}

extern "C" size_t bq_moe_route_backward_workspace_bytes(int32_t T, int32_t E) {
    if (T < 0 || T > kMaxRows || E < 1 || E > kMaxExperts) return 0;
    return up256((size_t)std::max(1, gradient_chunking(T, true).chunks) * E * 4);
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
    const Chunking c = gradient_chunking(T, dbias != nullptr);
    const bool one = dbias && T > 0 && T <= kOneClusterRows;
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
                          dtype, dbias ? static_cast<float*>(workspace) : nullptr, one ? dbias : nullptr, bq::device_status_ptr()};
    if (T > 0) {
        const size_t smem = dbias ? (size_t)kWarps * E * 4 : 0;
        const bool score = scoring == BQ_SCORE_SQRTSOFTPLUS;
        cudaError_t e = cudaSuccess;
        auto go = [&](auto constant, auto... more) {
            constexpr auto kernel = decltype(constant)::value;
            if ((e = allow_smem<kernel>(smem)) != cudaSuccess) return;
            if (one) e = launch_cluster(kernel, c.chunks, smem, st, a, more...);
            else e = bq::launch_after(kernel, dim3(c.chunks), dim3(kThreads), smem, st, a, more...);
        };
        if (dlosses) {
            const bool vec = E % 4 == 0 && bq::aligned(logits, 16) && bq::aligned(dlogits, 4 * es);
            with_share(E, vec, [&](auto nper, auto v) {
                constexpr int N = decltype(nper)::value;
                constexpr bool VEC = decltype(v)::value;
                score ? go(Constant<route_backward_kernel<N, VEC, RULE_SCORE>>()) : go(Constant<route_backward_kernel<N, VEC, RULE_SOFTMAX>>());
            });
        } else {
            const int wide = E * es % 16 == 0 && bq::aligned(dlogits, 16);
            score ? go(Constant<route_weights_backward_kernel<RULE_SCORE>>(), wide)
                  : go(Constant<route_weights_backward_kernel<RULE_SOFTMAX>>(), wide);
        }
        if ((s = launched(name, e)) != BQ_OK) return s;
    }
    if (!dbias || one) return BQ_OK;
    return launched(name, bq::launch_after(column_sums_kernel, dim3((E + 31) / 32), dim3(kThreads), 0, st,
                                           (const float*)workspace, T > 0 ? c.chunks : 0, E, dbias));
}
