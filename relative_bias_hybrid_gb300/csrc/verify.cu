// verify.cu -- the end of a verification step: the probabilities of rows of logits, and the drafts that
// stand with the token drawn behind them.
//
// [vLLM TML Inkling サポート, and vLLM hỗ trợ TML Inkling ..., the 8 chained MTP heads]: a decode step
// verifies the drafts of the heads.  Rejection sampling keeps the target's distribution: a draft x
// drawn from q stands with probability min(1, p(x) / q(x)), and the first that does not is
// replaced by a draw from max(p - q, 0), renormalised.
//
// k_token_probs: one row by the CTAs of a cluster.  A CTA's part of the row stays in registers between
// the maximum, the sum and the store, so the row is read once and written once; the CTAs exchange
// (maximum, sum) once through shared memory.  Rows of more than 8 x 32768 logits are read twice.
// Bound: HBM.
//
// k_verify_drafts: one sequence by the CTAs of a cluster.  Every CTA finds the first draft that does not
// stand (a few words), then sums its part of that one row; the other rows are never read.  Weights
// are whole multiples of 2^-43, so partial sums in 64 bits are exact: thread, warp, CTA and cluster sums
// nest, and the CTA, then the warp, then the lane in whose range the draw falls finds its token by
// the same sums.  Doubles would be exact too, but this part adds two a clock and SM: a row of 200000
// would take 11 us in doubles for 32 sequences, where reading it takes 8.
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace inkattn {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

// The 64-bit word at `local`'s offset in CTA `rank` of the cluster.
__device__ __forceinline__ void st_cluster_u64(uint32_t local, uint32_t rank, uint64_t v) {
    asm volatile("{\n\t.reg .b32 ra;\n\tmapa.shared::cluster.u32 ra, %0, %1;\n\t"
                 "st.shared::cluster.u64 [ra], %2;\n\t}" :: "r"(local), "r"(rank), "l"(v) : "memory");
}

// A row cut into groups of four elements at multiples of 16 bytes (bf16: 8), whatever its alignment:
// group g holds the elements 4 g - skew .. 4 g - skew + 3, the first and the last possibly in part.
__device__ __forceinline__ int row_skew(const void *row, int size) {
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
__device__ __forceinline__ float not_nan(float l) { return l == l ? l : -INFINITY; }

}  // namespace

// kPer = groups that a thread holds (a CTA's part is at most kThreads * kPer groups), 0: the part is
// read twice.
template <typename T, int kPer>
__global__ void __launch_bounds__(kThreads)
k_token_probs(const inkattn_token_probs_params p, int ctas) {
    __shared__ float s_red[kWarps];
    __shared__ int s_best;
    __shared__ __align__(8) uint64_t s_part[kMaxCluster];          // (maximum, sum or place) of each CTA
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = blockIdx.x / ctas, rank = blockIdx.x - row * ctas, V = p.V;
    const T *in = static_cast<const T *>(p.logits) + (size_t)row * p.logits_stride;
    float *out = p.probs + (size_t)row * p.probs_stride;
    const int skew = row_skew(in, sizeof(T));
    const bool same = skew == row_skew(out, 4);
    const int groups = (V + skew + 3) / 4, per = (groups + ctas - 1) / ctas;
    const int g0 = rank * per, g1 = min(groups, g0 + per);
    const float t = p.temperature ? load_f32(p.temperature + row) : 1.f;
    const bool valid = t >= 0.f && t < INFINITY, greedy = t == 0.f;
    if (!valid && rank == 0 && tid == 0) set_status(p.dev_status, INKATTN_ERR_DEVICE_BOUNDS);
    const float k = greedy ? 1.f : kLog2e / t;

    constexpr int kHold = kPer > 0 ? kPer : 1;
    float x[kHold][4];
    float m = -INFINITY, s = 0.f;
    if constexpr (kPer > 0) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int g = g0 + i * kThreads + tid;
            if (g < g1) load_group(in, 4 * g - skew, V, true, -INFINITY, x[i]);
            else x[i][0] = x[i][1] = x[i][2] = x[i][3] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) m = fmaxf(m, x[i][j]);     // (a NaN is passed over)
    } else {
        for (int g = g0 + tid; g < g1; g += kThreads) {
            load_group(in, 4 * g - skew, V, true, -INFINITY, x[0]);
            const float gm = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[0][2], x[0][3]));
            const float m2 = fmaxf(m, gm);
            s *= weight(m, m2, k);
            m = m2;
#pragma unroll
            for (int j = 0; j < 4; ++j) s += weight(not_nan(x[0][j]), m, k);
        }
    }
    const float m_thread = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) s_red[warp] = m;
    if (tid == 0) s_best = INT32_MAX;
    __syncthreads();
    m = s_red[lane & (kWarps - 1)];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    uint32_t second;                                               // this CTA's sum, or its best's place
    if (greedy) {
        int best = INT32_MAX;
        auto look = [&](int g, const float (&v)[4]) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (v[j] == m && (unsigned)(4 * g - skew + j) < (unsigned)V) best = min(best, 4 * g - skew + j);
        };
        if constexpr (kPer > 0) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int g = g0 + i * kThreads + tid;
                if (g < g1) look(g, x[i]);
            }
        } else if (m_thread == m) {
            for (int g = g0 + tid; g < g1; g += kThreads) {
                load_group(in, 4 * g - skew, V, true, -INFINITY, x[0]);
                look(g, x[0]);
            }
        }
        if (best != INT32_MAX) atomicMin(&s_best, best);
        __syncthreads();
        second = (uint32_t)s_best;
    } else {
        if constexpr (kPer > 0) {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[i][j] = weight(not_nan(x[i][j]), m, k);
                    s += x[i][j];
                }
        } else {
            s *= weight(m_thread, m, k);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        __syncthreads();
        if (lane == 0) s_red[warp] = s;
        __syncthreads();
        s = s_red[lane & (kWarps - 1)];
#pragma unroll
        for (int o = kWarps / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        second = __float_as_uint(s);
    }
    const uint64_t mine = ((uint64_t)__float_as_uint(m) << 32) | second;
    float m_all = m;
    if (ctas > 1) {
        if (tid < ctas) st_cluster_u64(smem_u32(&s_part[rank]), tid, mine);
        cluster_sync();
        for (int r = 0; r < ctas; ++r) m_all = fmaxf(m_all, __uint_as_float((uint32_t)(s_part[r] >> 32)));
    }
    // the row's sum, CTA by CTA in order, or the place of its first maximum
    int best = INT32_MAX;
    float sum = 0.f;
    for (int r = 0; r < ctas; ++r) {
        const uint64_t v = ctas > 1 ? s_part[r] : mine;
        const float mr = __uint_as_float((uint32_t)(v >> 32));
        if (greedy) {
            if (mr == m_all) best = min(best, (int)(uint32_t)v);
        } else {
            sum += weight(mr, m_all, k) * __uint_as_float((uint32_t)v);
        }
    }
    const bool zeros = !valid || m_all == -INFINITY;
    const float scale = zeros || greedy ? 0.f : 1.f / sum;
    const float scale_cta = scale * weight(m, m_all, k);           // of the weights held, which are against m
    auto store = [&](int g, const float (&v)[4]) {
        const int e = 4 * g - skew;
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            y[j] = zeros ? 0.f : greedy ? (e + j == best ? 1.f : 0.f) : kPer > 0 ? v[j] * scale_cta
                 : weight(not_nan(v[j]), m_all, k) * scale;
        if (same && e >= 0 && e + 4 <= V) {
            *reinterpret_cast<float4 *>(out + e) = make_float4(y[0], y[1], y[2], y[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if ((unsigned)(e + j) < (unsigned)V) out[e + j] = y[j];
        }
    };
    if constexpr (kPer > 0) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int g = g0 + i * kThreads + tid;
            if (g < g1) store(g, x[i]);
        }
    } else {
        for (int g = g0 + tid; g < g1; g += kThreads) {
            load_group(in, 4 * g - skew, V, true, -INFINITY, x[0]);
            store(g, x[0]);
        }
    }
}

// CTAs of a row: enough that a CTA's part fits its registers eight groups a thread, more where the rows
// alone do not fill the GPU (a part then has at least a group for each thread).
cudaError_t launch_token_probs(const inkattn_token_probs_params &p, int num_sms, cudaStream_t stream) {
    const int groups = p.V / 4 + 2;
    int ctas = 1;
    while (ctas < kMaxCluster && (groups > 8 * kThreads * ctas ||
                                  ((long long)p.N_tok * ctas < 2 * num_sms && groups > kThreads * ctas)))
        ctas *= 2;
    const int per = (groups + ctas - 1) / ctas;
    auto kernel = [&](auto type) {
        using T = decltype(type);
        return per <= 8 * kThreads ? k_token_probs<T, 8> : per <= 16 * kThreads ? k_token_probs<T, 16> : k_token_probs<T, 0>;
    };
    return launch_dependent(p.logits_dtype == INKATTN_DTYPE_F32 ? kernel(0.f) : kernel(inkattn_bf16{}),
                            dim3((unsigned)(p.N_tok * ctas)), dim3(kThreads), 0, stream, ctas, p, ctas);
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

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace

__global__ void __launch_bounds__(kThreads)
k_verify_drafts(const inkattn_verify_drafts_params p, int ctas) {
    __shared__ int s_accepted;
    __shared__ uint64_t s_warp[kWarps];
    __shared__ __align__(8) uint64_t s_total[2][kMaxCluster];
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = blockIdx.x / ctas, rank = blockIdx.x - b * ctas, V = p.V;
    const int start = load_i32(p.cu_seqlens_q + b), end = load_i32(p.cu_seqlens_q + b + 1);
    const bool bad = start < 0 || end < start || end > p.N_tok;
    if (bad || start == end) {                         // (the same in every CTA of the cluster)
        if (rank == 0 && tid == 0) {
            if (bad) set_status(p.dev_status, INKATTN_ERR_DEVICE_BOUNDS);
            p.n_new[b] = 0;
        }
        return;
    }
    const int n = end - start, drafts = n - 1;

    // ---- the first draft that does not stand
    if (warp == 0) {
        int accepted = drafts;
        for (int base = 0; base < drafts; base += 32) {
            const int i = base + lane;
            bool stands = true;
            if (i < drafts) {
                const size_t row = (size_t)start + i;
                const int x = load_i32(p.token_ids + row + 1);
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
                break;
            }
        }
        if (lane == 0) s_accepted = accepted;
    }
    __syncthreads();
    const int accepted = s_accepted;

    // ---- the weights of the row behind the drafts that stand
    const size_t row = (size_t)start + accepted;
    const float *pr = p.target_p + row * p.target_stride;
    const float *qr = nullptr;
    int without = -1;                                  // the token left out (a draft without choice)
    if (accepted < drafts) {
        const int x = load_i32(p.token_ids + row + 1);
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
    auto weights = [&](int g, float (&w)[4]) {
        const int e = 4 * g - skew;
        load_group(pr, e, V, true, 0.f, w);
        float q[4] = {0.f, 0.f, 0.f, 0.f};
        if (qr) load_group(qr, e, V, row_skew(qr, 4) == skew, 0.f, q);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = e + j == without ? 0.f : fmaxf(unit(w[j]) - unit(q[j]), 0.f);
    };
    uint64_t total = 0;
    int round = 0;
    for (;; ++round) {
        uint32_t hi = 0, lo = 0;                       // (at most 256 weights a thread: below 2^31)
#pragma unroll 4
        for (int g = g0 + lane; g < g1; g += 32) {
            float w[4];
            weights(g, w);
#pragma unroll
            for (int j = 0; j < 4; ++j) fixed_add(w[j], hi, lo);
        }
        const uint64_t mine = warp_sum(((uint64_t)hi << 22) + lo);
        if (lane == 0) s_warp[warp] = mine;
        __syncthreads();
        uint64_t cta = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) cta += s_warp[i];
        if (ctas > 1) {
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
    if (rank == 0) {
        for (int i = tid; i < n; i += kThreads) {
            if (i < accepted) p.out_tokens[start + i] = load_i32(p.token_ids + start + i + 1);
            else if (i > accepted || total == 0) p.out_tokens[start + i] = -1;
        }
        if (tid == 0) {
            p.n_new[b] = accepted + (total != 0 ? 1 : 0);
            if (total == 0) set_status(p.dev_status, INKATTN_ERR_DEVICE_BOUNDS);
        }
    }
    if (total == 0) return;
    const uint64_t u = (uint64_t)(below_one(load_f32(p.u_sample + b)) * 0x1p32f);
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
    for (int base = g0; base < g1; base += 32) {       // (one warp of the cluster is left)
        const int g = base + lane;
        uint64_t step[4] = {0, 0, 0, 0}, upto = 0;
        if (g < g1) {
            float w[4];
            weights(g, w);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t hi = 0, lo = 0;
                fixed_add(w[j], hi, lo);
                step[j] = ((uint64_t)hi << 22) + lo;
                upto += step[j];
            }
        }
        const uint64_t own = upto;
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
        if (rest < upto && rest >= upto - own) {       // this lane's group
            uint64_t left = rest - (upto - own);
            int j = 0;
            while (j < 3 && left >= step[j]) left -= step[j++];
            p.out_tokens[row] = 4 * g - skew + j;
        }
        break;
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
