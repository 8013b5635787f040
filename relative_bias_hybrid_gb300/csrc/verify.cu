// verify.cu -- the end of a verification step: the probabilities of rows of logits, and the drafts that
// stand with the token drawn behind them.
//
// [vLLM TML Inkling サポート, and vLLM hỗ trợ TML Inkling ..., the 8 chained MTP heads]: a decode step
// verifies the drafts of the heads.  Rejection sampling keeps the target's distribution: a draft x
// drawn from q stands with probability min(1, p(x) / q(x)), and the first that does not is
// replaced by a draw from max(p - q, 0), renormalised.
//
// k_token_probs: one row by the CTAs of a cluster, which exchange (maximum, sum) once through shared
// memory.  Where all clusters are resident at once, a CTA's part of the row stays in registers
// between the maximum, the sum and the store (k_token_probs: few rows, bound by the chain of these
// steps: 9 rows of 50001 bf16 logits 5.3 us, read twice 9.3).  Otherwise the row is read again for the
// store, from L2 (k_token_probs_twice): a thread then holds nothing over the exchange and
// four CTAs an SM keep loading, where parts held in registers let two, in step (288 rows of
// 131072 fp32 logits: 58 us, 5.2 TB/s to and from HBM; held in registers 140, and 93 with each
// thread's next row on its way into shared memory meanwhile).  Steps: 66 us with every element tested for
// the row's end and for an infinite maximum (49 warp instructions for 32 logits, now 28) 60, and with
// stores that leave L2 first 58.
//
// k_verify_drafts: one sequence by the CTAs of a cluster.  Every CTA finds the first draft that does not
// stand (a few words), then sums its part of that one row; the other rows are never read.  Weights
// are whole multiples of 2^-43, so partial sums in 64 bits are exact: thread, warp, CTA and cluster sums
// nest, and the CTA, then the warp, then the lane in whose range the draw falls finds its token by
// the same sums.  (Doubles keep the sums as well, but an SM adds two a clock: 32 rows of 200000 would take
// 11 us, where reading them from HBM takes 8.)  One sequence over 131072 tokens 7.0 us, of which the
// launch and four dependent round trips to memory are nearly all; 32 over 200019 14.3 us, 3.6 TB/s (19.8
// with the loads of one group at a time and the whole of the last warp's part read again).
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace inkattn {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kPer = 8;                    // groups of four that a thread of k_token_probs holds

// The 64-bit word at `local`'s offset in CTA `rank` of the cluster.
__device__ __forceinline__ void st_cluster_u64(uint32_t local, uint32_t rank, uint64_t v) {
    asm volatile("{\n\t.reg .b32 ra;\n\tmapa.shared::cluster.u32 ra, %0, %1;\n\t"
                 "st.shared::cluster.u64 [ra], %2;\n\t}" :: "r"(local), "r"(rank), "l"(v) : "memory");
}

// A row cut into groups of four elements at multiples of 16 bytes (bf16: 8), whatever its alignment:
// group g holds the elements 4 g - skew .. 4 g - skew + 3, the first and the last possibly in part.
__host__ __device__ __forceinline__ int row_skew(const void *row, int size) {
    return (int)((reinterpret_cast<uintptr_t>(row) / size) & 3);
}
template <typename T>
__device__ __forceinline__ float load_one(const T *p) {
    if constexpr (std::is_same<T, float>::value) return load_f32(p);
    unsigned short v;
    asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(reinterpret_cast<uint64_t>(p)));
    return __uint_as_float((uint32_t)v << 16);
}
template <typename T>
__device__ __forceinline__ void load_four(const T *p, float (&x)[4]) {
    if constexpr (std::is_same<T, float>::value) {
        const uint4 v = load_u32x4(p);
        x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
    } else {
        uint32_t a, b;
        asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "l"(reinterpret_cast<uint64_t>(p)));
        x[0] = bf16_lo(a); x[1] = bf16_hi(a);
        x[2] = bf16_lo(b); x[3] = bf16_hi(b);
    }
}
// Elements e .. e + 3 of a row of V, `none` outside it; together: in one access (an aligned group).
template <typename T>
__device__ __forceinline__ void load_group(const T *row, int e, int V, bool together, float none, float (&x)[4]) {
    if (together && e >= 0 && e + 4 <= V) {
        load_four(row + e, x);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = (unsigned)(e + j) < (unsigned)V ? load_one(row + e + j) : none;
    }
}

// ---------------------------------------------------------------- probabilities

// exp((l - m) k / log2 e) for l <= m; 1 at the maximum (also an infinite one), 0 for -infinity
__device__ __forceinline__ float weight(float l, float m, float k) {
    return l == -INFINITY ? 0.f : l == m ? 1.f : fast_exp2((l - m) * k);
}
// Logits to their weights, a NaN as -infinity; m is their maximum or larger.  (k is finite, so an infinite
// m alone needs the comparisons.)
__device__ __forceinline__ void to_weights(float (&x)[4], float m, float k) {
    if (m < INFINITY) {
        const float below = m == -INFINITY ? 0.f : -m;
        const float2 a = fmul2(fadd2(make_float2(x[0], x[1]), make_float2(below, below)), make_float2(k, k));
        const float2 b = fmul2(fadd2(make_float2(x[2], x[3]), make_float2(below, below)), make_float2(k, k));
        x[0] = fast_exp2(fmaxf(a.x, -INFINITY));
        x[1] = fast_exp2(fmaxf(a.y, -INFINITY));
        x[2] = fast_exp2(fmaxf(b.x, -INFINITY));
        x[3] = fast_exp2(fmaxf(b.y, -INFINITY));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = weight(fmaxf(x[j], -INFINITY), m, k);
    }
}
// log2(e) / t, finite also for the smallest t; 1 for a greedy row (t = 0)
__device__ __forceinline__ float exponent_factor(float t) { return t == 0.f ? 1.f : fminf(kLog2e / t, 0x1.fffffep127f); }

// What the CTAs of a row know of it.
template <typename T>
struct RowPart {
    const T *in;
    float *out;
    int skew, g0, g1;                      // this CTA's groups
    bool same;                             // in and out are aligned alike
};
template <typename T>
__device__ __forceinline__ RowPart<T> row_part(const inkattn_token_probs_params &p, int row, int rank, int ctas) {
    RowPart<T> r;
    r.in = static_cast<const T *>(p.logits) + (size_t)row * p.logits_stride;
    r.out = p.probs + (size_t)row * p.probs_stride;
    r.skew = row_skew(r.in, sizeof(T));
    r.same = r.skew == row_skew(r.out, 4);
    const int groups = (p.V + r.skew + 3) / 4, per = (groups + ctas - 1) / ctas;
    r.g0 = rank * per;
    r.g1 = min(groups, r.g0 + per);
    return r;
}
template <typename T>
__device__ __forceinline__ void store_group(const RowPart<T> &r, int e, int V, const float (&y)[4]) {
    if (r.same && e >= 0 && e + 4 <= V) {
        *reinterpret_cast<float4 *>(r.out + e) = make_float4(y[0], y[1], y[2], y[3]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if ((unsigned)(e + j) < (unsigned)V) r.out[e + j] = y[j];
    }
}

// The maximum of a block's values; the sum of a block's values (in a fixed order).
__device__ __forceinline__ float block_max(float m, float *s_red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = m;
    __syncthreads();
    m = s_red[threadIdx.x & (kWarps - 1)];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}
__device__ __forceinline__ float block_sum(float s, float *s_red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    __syncthreads();                       // (s_red held the maxima)
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = s;
    __syncthreads();
    s = s_red[threadIdx.x & (kWarps - 1)];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// The row's maximum and sum, CTA by CTA in order, or the place of its first maximum, from every CTA's
// (maximum, sum or place).
struct RowTotal {
    float m, sum;
    int best;
};
__device__ __forceinline__ RowTotal row_total(float m, uint32_t second, bool greedy, float k, int rank, int ctas,
                                              uint64_t *s_part) {
    const uint64_t mine = ((uint64_t)__float_as_uint(m) << 32) | second;
    RowTotal t = {m, 0.f, INT32_MAX};
    if (ctas > 1) {
        cluster_started_wait();
        if ((int)threadIdx.x < ctas) st_cluster_u64(smem_u32(&s_part[rank]), threadIdx.x, mine);
        cluster_sync();
        for (int r = 0; r < ctas; ++r) t.m = fmaxf(t.m, __uint_as_float((uint32_t)(s_part[r] >> 32)));
    }
    for (int r = 0; r < ctas; ++r) {
        const uint64_t v = ctas > 1 ? s_part[r] : mine;
        const float mr = __uint_as_float((uint32_t)(v >> 32));
        if (greedy) {
            if (mr == t.m) t.best = min(t.best, (int)(uint32_t)v);
        } else {
            t.sum += weight(mr, t.m, k) * __uint_as_float((uint32_t)v);
        }
    }
    return t;
}

}  // namespace

// A CTA's part of a row is at most kThreads * kPer groups.
template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
k_token_probs(const inkattn_token_probs_params p, int ctas) {
    __shared__ float s_red[kWarps];
    __shared__ int s_best;
    __shared__ __align__(8) uint64_t s_part[kMaxCluster];
    grid_dep_wait();
    grid_dep_launch();
    if (ctas > 1) cluster_started_arrive();
    const int tid = threadIdx.x, V = p.V;
    const int row = blockIdx.x / ctas, rank = blockIdx.x - row * ctas;
    const RowPart<T> r = row_part<T>(p, row, rank, ctas);
    const float t = p.temperature ? load_f32(p.temperature + row) : 1.f;
    float x[kPer][4], m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int g = r.g0 + i * kThreads + tid;
        if (g < r.g1) load_group(r.in, 4 * g - r.skew, V, true, -INFINITY, x[i]);
        else x[i][0] = x[i][1] = x[i][2] = x[i][3] = -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) m = fmaxf(m, x[i][j]);         // (a NaN is passed over)
    const bool valid = t >= 0.f && t < INFINITY, greedy = t == 0.f;
    if (!valid && rank == 0 && tid == 0) set_status(p.dev_status, INKATTN_ERR_DEVICE_BOUNDS);
    const float k = exponent_factor(t);
    if (tid == 0) s_best = INT32_MAX;
    m = block_max(m, s_red);
    uint32_t second;                                               // this CTA's sum, or its first maximum's place
    if (greedy) {
        int best = INT32_MAX;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int g = r.g0 + i * kThreads + tid, e = 4 * g - r.skew + j;
                if (x[i][j] == m && g < r.g1 && (unsigned)e < (unsigned)V) best = min(best, e);
            }
        if (best != INT32_MAX) atomicMin(&s_best, best);
        __syncthreads();
        second = (uint32_t)s_best;
    } else {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            to_weights(x[i], m, k);
            s += (x[i][0] + x[i][1]) + (x[i][2] + x[i][3]);
        }
        second = __float_as_uint(block_sum(s, s_red));
    }
    const RowTotal total = row_total(m, second, greedy, k, rank, ctas, s_part);
    const bool zeros = !valid || total.m == -INFINITY;
    // of the weights held, which are against this CTA's maximum
    const float scale = zeros || greedy ? 0.f : weight(m, total.m, k) / total.sum;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int g = r.g0 + i * kThreads + tid, e = 4 * g - r.skew;
        if (g >= r.g1) break;
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = zeros ? 0.f : greedy ? (e + j == total.best ? 1.f : 0.f) : x[i][j] * scale;
        store_group(r, e, V, y);
    }
}

// Four groups at a time: their loads go out together.
template <typename T>
__global__ void __launch_bounds__(kThreads, 4)
k_token_probs_twice(const inkattn_token_probs_params p, int ctas) {
    __shared__ float s_red[kWarps];
    __shared__ int s_best;
    __shared__ __align__(8) uint64_t s_part[kMaxCluster];
    grid_dep_wait();
    grid_dep_launch();
    if (ctas > 1) cluster_started_arrive();
    const int tid = threadIdx.x, V = p.V;
    const int row = blockIdx.x / ctas, rank = blockIdx.x - row * ctas;
    const RowPart<T> r = row_part<T>(p, row, rank, ctas);
    const float t = p.temperature ? load_f32(p.temperature + row) : 1.f;
    const bool valid = t >= 0.f && t < INFINITY, greedy = t == 0.f;
    if (!valid && rank == 0 && tid == 0) set_status(p.dev_status, INKATTN_ERR_DEVICE_BOUNDS);
    const float k = exponent_factor(t);
    constexpr int kAhead = 4;
    // whether a thread's next groups, from g on, are all there and whole
    auto whole = [&](int g) {
        const int e = 4 * g - r.skew;
        return g + (kAhead - 1) * kThreads < r.g1 && e >= 0 && e + 4 * (kAhead - 1) * kThreads + 4 <= V;
    };
    auto load = [&](int g, float (&x)[kAhead][4]) {
        if (whole(g)) {
            const T *at = r.in + (4 * g - r.skew);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) load_four(at + 4 * i * kThreads, x[i]);
            return;
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int gi = g + i * kThreads;
            if (gi < r.g1) load_group(r.in, 4 * gi - r.skew, V, true, -INFINITY, x[i]);
            else x[i][0] = x[i][1] = x[i][2] = x[i][3] = -INFINITY;
        }
    };
    float m = -INFINITY, s = 0.f;
    for (int g = r.g0 + tid; g < r.g1; g += kAhead * kThreads) {
        float x[kAhead][4];
        load(g, x);
        float m2 = m;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) m2 = fmaxf(m2, fmaxf(fmaxf(x[i][0], x[i][1]), fmaxf(x[i][2], x[i][3])));
        s *= weight(m, m2, k);
        m = m2;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            to_weights(x[i], m, k);
            s += (x[i][0] + x[i][1]) + (x[i][2] + x[i][3]);
        }
    }
    const float m_thread = m;
    if (tid == 0) s_best = INT32_MAX;
    m = block_max(m, s_red);
    uint32_t second;
    if (greedy) {
        int best = INT32_MAX;
        if (m_thread == m) {
            for (int g = r.g0 + tid; g < r.g1; g += kThreads) {
                float x[4];
                load_group(r.in, 4 * g - r.skew, V, true, -INFINITY, x);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (x[j] == m && (unsigned)(4 * g - r.skew + j) < (unsigned)V) best = min(best, 4 * g - r.skew + j);
            }
        }
        if (best != INT32_MAX) atomicMin(&s_best, best);
        __syncthreads();
        second = (uint32_t)s_best;
    } else {
        second = __float_as_uint(block_sum(s * weight(m_thread, m, k), s_red));
    }
    const RowTotal total = row_total(m, second, greedy, k, rank, ctas, s_part);
    const bool zeros = !valid || total.m == -INFINITY;
    const float scale = zeros || greedy ? 0.f : 1.f / total.sum;
    for (int g = r.g0 + tid; g < r.g1; g += kAhead * kThreads) {
        float x[kAhead][4];
        if (!greedy && !zeros) {
            load(g, x);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                to_weights(x[i], total.m, k);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[i][j] *= scale;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    x[i][j] = !zeros && 4 * (g + i * kThreads) - r.skew + j == total.best ? 1.f : 0.f;
        }
        if (r.same && whole(g)) {
            float *at = r.out + (4 * g - r.skew);
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                __stcs(reinterpret_cast<float4 *>(at + 4 * i * kThreads), make_float4(x[i][0], x[i][1], x[i][2], x[i][3]));
        } else {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (g + i * kThreads >= r.g1) break;
                store_group(r, 4 * (g + i * kThreads) - r.skew, V, x[i]);
            }
        }
    }
}

namespace {

template <typename T>
cudaError_t launch_token_probs_of(const inkattn_token_probs_params &p, int num_sms, cudaStream_t stream) {
    // the most groups of a row: those of every row where all are aligned alike
    const int skew = p.logits_stride % 4 == 0 || p.N_tok == 1 ? row_skew(p.logits, sizeof(T)) : 3;
    const int groups = (p.V + skew + 3) / 4;
    // CTAs of a row: a part of at most 64 KB (288 rows of 131072 fp32: 58 us, parts of 128 KB 64, of 256 KB
    // 77; bf16 45, parts of 32 KB 50, and 50001 20, parts of 25 KB 27: a CTA's fixed cost is about 5 us), and
    // more CTAs as long as all are resident at once and a part has a group for each thread (64 rows of
    // 50001 bf16 with four 8.0 us, two 9.4, eight 11.4)
    constexpr int kMost = 65536 / (4 * (int)sizeof(T));
    int ctas = 1;
    while (ctas < kMaxCluster &&
           (groups > kMost * ctas || ((long long)p.N_tok * ctas <= num_sms && groups > kThreads * ctas)))
        ctas *= 2;
    const bool few = (long long)p.N_tok * ctas <= 2 * num_sms && (groups + ctas - 1) / ctas <= kPer * kThreads;
    return launch_dependent(few ? k_token_probs<T> : k_token_probs_twice<T>, dim3((unsigned)(p.N_tok * ctas)),
                            dim3(kThreads), 0, stream, ctas, p, ctas);
}

}  // namespace

cudaError_t launch_token_probs(const inkattn_token_probs_params &p, int num_sms, cudaStream_t stream) {
    return p.logits_dtype == INKATTN_DTYPE_F32 ? launch_token_probs_of<float>(p, num_sms, stream)
                                               : launch_token_probs_of<inkattn_bf16>(p, num_sms, stream);
}

// ---------------------------------------------------------------- verification

namespace {

__device__ __forceinline__ float unit(float v) { return fminf(fmaxf(v, 0.f), 1.f); }               // NaN: 0
__device__ __forceinline__ float below_one(float u) { return fminf(fmaxf(u, 0.f), 0x1.fffffep-1f); }

// A weight in [0, 1] in steps of 2^-43, rounded to nearest, ties to even: steps = hi 2^22 + lo.
// w + 4, rounded down, ends at 2^-21 and so counts its multiples in the mantissa; the rest, exact, plus
// 2^-20 ends at 2^-43 and counts those.  Ten instructions without a conversion.
__device__ __forceinline__ void fixed_add(float w, uint32_t &hi, uint32_t &lo) {
    const float h = __fadd_rz(w, 4.f);
    const float l = __fadd_rn(w - (h - 4.f), 0x1p-20f);
    hi += __float_as_uint(h) - 0x40800000u;
    lo += __float_as_uint(l) - 0x35800000u;
}

constexpr int kAhead = 4;                  // groups of a lane that are asked for together: a batch
// batches of a warp for the longest vocabulary
constexpr int kMaxBatches = (INKATTN_MAX_VOCAB / 4 + 2 + kMaxCluster * kWarps * 32 * kAhead - 1) / (kMaxCluster * kWarps * 32 * kAhead) + 1;

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace

__global__ void __launch_bounds__(kThreads)
k_verify_drafts(const inkattn_verify_drafts_params p, int ctas) {
    __shared__ int s_accepted, s_lost;
    __shared__ uint64_t s_warp[kWarps], s_batch[kWarps][kMaxBatches];
    __shared__ __align__(8) uint64_t s_total[2][kMaxCluster];
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = blockIdx.x / ctas, rank = blockIdx.x - b * ctas, V = p.V;
    const int start = load_i32(p.cu_seqlens_q + b), end = load_i32(p.cu_seqlens_q + b + 1);
    const float u_sample = load_f32(p.u_sample + b);   // (needed last, asked for first)
    const bool bad = start < 0 || end < start || end > p.N_tok;
    if (bad || start == end) {                         // (the same in every CTA of the cluster)
        if (rank == 0 && tid == 0) {
            if (bad) set_status(p.dev_status, INKATTN_ERR_DEVICE_BOUNDS);
            p.n_new[b] = 0;
        }
        return;
    }
    if (ctas > 1) cluster_started_arrive();
    const int n = end - start, drafts = n - 1;

    // ---- the first draft that does not stand
    if (warp == 0) {
        int accepted = drafts;
        for (int base = 0; base < drafts; base += 32) {
            const int i = base + lane;
            bool stands = true;
            int x = 0;
            if (i < drafts) {
                const size_t row = (size_t)start + i;
                x = load_i32(p.token_ids + row + 1);
                stands = false;
                if (x >= 0 && x < V) {
                    const float u = below_one(load_f32(p.u_accept + row));
                    const float pt = unit(load_f32(p.target_p + row * p.target_stride + x));
                    const float q = p.draft_p ? unit(load_f32(p.draft_p + row * p.draft_stride + x)) : 1.f;
                    stands = __fmul_rn(u, q) < pt;
                }
            }
            const uint32_t no = __ballot_sync(0xffffffffu, !stands);
            if (no) {
                accepted = base + __ffs(no) - 1;
                if (i == accepted) s_lost = x;
                break;
            }
        }
        if (lane == 0) s_accepted = accepted;
    }
    __syncthreads();
    const int accepted = s_accepted;
    if (rank == 0)
        for (int i = tid; i < n; i += kThreads)
            if (i != accepted) p.out_tokens[start + i] = i < accepted ? load_i32(p.token_ids + start + i + 1) : -1;

    // ---- the weights of the row behind the drafts that stand
    const size_t row = (size_t)start + accepted;
    const float *pr = p.target_p + row * p.target_stride;
    const float *qr = nullptr;
    int without = -1;                                  // the token left out (a draft without choice)
    if (accepted < drafts) {
        const int x = s_lost;
        if (x < 0 || x >= V) {
            if (rank == 0 && tid == 0) set_status(p.dev_status, INKATTN_ERR_DEVICE_BOUNDS);
        } else if (p.draft_p) {
            qr = p.draft_p + row * p.draft_stride;
        } else {
            without = x;
        }
    }
    const int skew = row_skew(pr, 4);
    const int groups = (V + skew + 3) / 4, per = (groups + ctas - 1) / ctas, per_warp = (per + kWarps - 1) / kWarps;
    const int g0 = min(groups, rank * per + warp * per_warp);
    const int g1 = min(min(groups, rank * per + per), g0 + per_warp);
    // the weights of this lane's groups at g, g + 32, ..., kAhead of them: their loads go out together
    auto weights = [&](int g, float (&w)[kAhead][4]) {
        const bool together = qr && row_skew(qr, 4) == skew;
        float q[kAhead][4];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int gi = g + 32 * i, e = 4 * gi - skew;
#pragma unroll
            for (int j = 0; j < 4; ++j) w[i][j] = q[i][j] = 0.f;
            if (gi < g1) {
                load_group(pr, e, V, true, 0.f, w[i]);
                if (qr) load_group(qr, e, V, together, 0.f, q[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[i][j] = 4 * (g + 32 * i) - skew + j == without ? 0.f : fmaxf(unit(w[i][j]) - unit(q[i][j]), 0.f);
    };
    uint64_t total = 0;
    int round = 0;
    for (;; ++round) {
        uint64_t mine = 0;                             // the warp's sum, and that of each batch of loads
        for (int base = g0, batch = 0; base < g1; base += 32 * kAhead, ++batch) {
            float w[kAhead][4];
            weights(base + lane, w);
            uint32_t hi = 0, lo = 0;
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) fixed_add(w[i][j], hi, lo);
            const uint64_t sum = warp_sum(((uint64_t)hi << 22) + lo);
            if (lane == 0) s_batch[warp][batch] = sum;
            mine += sum;
        }
        if (lane == 0) s_warp[warp] = mine;
        __syncthreads();
        uint64_t cta = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) cta += s_warp[i];
        if (ctas > 1) {
            if (round == 0) cluster_started_wait();
            if (tid < ctas) st_cluster_u64(smem_u32(&s_total[round][rank]), tid, cta);
            cluster_sync();
        } else {
            if (tid == 0) s_total[round][0] = cta;
            __syncthreads();
        }
        for (int r = 0; r < ctas; ++r) total += s_total[round][r];
        if (total != 0 || round == 1 || (!qr && without < 0)) break;
        qr = nullptr;                                  // p nowhere above q: from p itself
        without = -1;
    }

    // ---- the draw
    if (rank == 0 && tid == 0) {
        p.n_new[b] = accepted + (total != 0 ? 1 : 0);
        if (total == 0) {
            p.out_tokens[row] = -1;
            set_status(p.dev_status, INKATTN_ERR_DEVICE_BOUNDS);
        }
    }
    if (total == 0) return;
    const uint64_t u = (uint64_t)(below_one(u_sample) * 0x1p32f);
    uint64_t rest = __umul64hi(total, u << 32);        // floor(W U / 2^32) < W
    for (int r = 0; r < rank; ++r) {
        if (rest < s_total[round][r]) return;          // an earlier CTA's
        rest -= s_total[round][r];
    }
    if (rest >= s_total[round][rank]) return;
    for (int i = 0; i < warp; ++i) {
        if (rest < s_warp[i]) return;
        rest -= s_warp[i];
    }
    if (rest >= s_warp[warp]) return;
    // one warp of the cluster is left; its batch, read again, has the token
    for (int base = g0, batch = 0; base < g1; base += 32 * kAhead, ++batch) {
        if (rest >= s_batch[warp][batch]) {
            rest -= s_batch[warp][batch];
            continue;
        }
        float w[kAhead][4];
        weights(base + lane, w);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            uint64_t step[4], own = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t hi = 0, lo = 0;
                fixed_add(w[i][j], hi, lo);
                step[j] = ((uint64_t)hi << 22) + lo;
                own += step[j];
            }
            uint64_t upto = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            const uint64_t all = __shfl_sync(0xffffffffu, upto, 31);
            if (rest >= all) {
                rest -= all;
                continue;
            }
            if (rest < upto && rest >= upto - own) {               // this lane's group
                uint64_t left = rest - (upto - own);
                int j = 0;
#pragma unroll
                for (int c = 0; c < 3; ++c)
                    if (j == c && left >= step[c]) {
                        left -= step[c];
                        ++j;
                    }
                p.out_tokens[row] = 4 * (base + lane + 32 * i) - skew + j;
            }
            return;
        }
    }
}

// CTAs of a sequence: a group for each thread at least, eight CTAs at most.
cudaError_t launch_verify_drafts(const inkattn_verify_drafts_params &p, cudaStream_t stream) {
    const int groups = p.V / 4 + 2;
    int ctas = 1;
    while (ctas < kMaxCluster && groups > kThreads * ctas) ctas *= 2;
    return launch_dependent(k_verify_drafts, dim3((unsigned)(p.B * ctas)), dim3(kThreads), 0, stream, ctas, p, ctas);
}

}  // namespace inkattn
