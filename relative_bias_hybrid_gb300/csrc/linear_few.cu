// linear_few.cu -- linear layers of few tokens, or small ones, without the tensor cores.
//
// out[t][f] = act( sum_k x[t][k] w[f][k] + bias[f] ) + residual[t][f]
//
// [vLLM hỗ trợ TML Inkling ..., §TP sharding nhận biết sconv]: the output projection of a decode
//  step.
//
// Bound by the weights, which are read once: a single user's step has few products for each
// byte of them, which fp32 multiply-adds keep up with, and what the tensor-core kernel
// (linear.cu) needs before its first product (TMEM, descriptors, a ring, a cluster) is most of its
// time for small layers.  A group of one, four or sixteen warps takes two weight rows (SWIGLU: a
// gate row and the up row of the same feature), or four for more than four tokens; a thread has pieces
// of 8 values (16 bytes) of the rows in turn, four of each requested together, and multiplies them
// with the same pieces of every token, which come from L1.  Sums are held in fp32, in pairs; the
// threads' sums are added in a fixed order, by halves within a warp, then warp by warp.
//
// Measured, where the tensor-core kernel takes the time in brackets: 1 token 1024 x 1024 1.9 us (4.2),
// 8192 x 258 2.5 (8.3), 8192 x 4096 12.3 (15.3), 8192 x 8192 22.9 (23.6), 5.9 TB/s; 4 tokens 4096 x
// 2048 6.9 (7.6); 8 tokens 2048 x 2048 5.6 (6.0).  More tokens cost it more: with x from L1 and
// fewer threads an SM, 8 tokens 8192 x 8192 39 us (23.7).
#include <type_traits>

#include "activation.cuh"
#include "common.cuh"
#include "internal.h"

namespace inkattn {

namespace {

__host__ __device__ constexpr int rows_of_group(int tok) { return tok > 4 ? 4 : 2; }   // weight rows
constexpr int kU = 4;                              // pieces of a row requested together
constexpr int kMostTokens = 256;
constexpr int kFewThreads = 128;                   // of a block, or one group of more

template <bool kExact>
__device__ __forceinline__ float activate_any(int act, float v) {
    switch (act) {
        case INKATTN_ACT_RELU: return activate<INKATTN_ACT_RELU, kExact>(v);
        case INKATTN_ACT_GELU: return activate<INKATTN_ACT_GELU, kExact>(v);
        case INKATTN_ACT_SILU: case INKATTN_ACT_SWIGLU: return activate<INKATTN_ACT_SILU, kExact>(v);
        default: return v;
    }
}

}  // namespace

// kTok: tokens of a block, or more; kWarps: warps of a group.  Tokens behind the last and rows behind the last
// feature read the last one's and are not stored.
template <int kTok, int kWarps>
__global__ void __launch_bounds__(kWarps * 32 > kFewThreads ? kWarps * 32 : kFewThreads)
k_linear_few(const LinearArgs A, int act) {
    constexpr int kThreads = kWarps * 32 > kFewThreads ? kWarps * 32 : kFewThreads;
    constexpr int kGroups = kThreads / (kWarps * 32);      // of a block
    constexpr int kR = rows_of_group(kTok), kN = kR * kTok;
    __shared__ float s_part[kThreads / 32][kN];
    grid_dep_wait();
    grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = (int)blockIdx.x * kGroups + warp / kWarps;
    const bool gated = act == INKATTN_ACT_SWIGLU;
    const int feats = gated ? kR / 2 : kR, f0 = group * feats;
    const int pieces = A.K >> 3, t0 = (int)blockIdx.y * kTok;
    const uint4 *w[kR], *x[kTok];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
        const int f = min(f0 + (gated ? r % (kR / 2) : r), A.F - 1);
        w[r] = reinterpret_cast<const uint4 *>(A.w) + ((size_t)f + (gated && r >= kR / 2 ? (size_t)A.F : 0)) * pieces;
    }
#pragma unroll
    for (int t = 0; t < kTok; ++t) x[t] = reinterpret_cast<const uint4 *>(A.x) + (size_t)min(t0 + t, A.M - 1) * pieces;
    float2 acc[kR][kTok] = {};
    constexpr int kStep = kWarps * 32;
    for (int p0 = (warp % kWarps) * 32 + lane; p0 < pieces; p0 += kStep * kU) {
        uint4 v[kU][kR];
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                v[u][r] = make_uint4(0, 0, 0, 0);
                if (p0 + u * kStep < pieces) v[u][r] = __ldcs(w[r] + p0 + u * kStep);
            }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (p0 + u * kStep >= pieces) break;
#pragma unroll
            for (int t = 0; t < kTok; ++t) {
                const uint4 q = x[t][p0 + u * kStep];
                const float2 x0 = make_float2(bf16_lo(q.x), bf16_hi(q.x)), x1 = make_float2(bf16_lo(q.y), bf16_hi(q.y));
                const float2 x2 = make_float2(bf16_lo(q.z), bf16_hi(q.z)), x3 = make_float2(bf16_lo(q.w), bf16_hi(q.w));
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    const uint4 m = v[u][r];
                    float2 s = acc[r][t];
                    s = ffma2(make_float2(bf16_lo(m.x), bf16_hi(m.x)), x0, s);
                    s = ffma2(make_float2(bf16_lo(m.y), bf16_hi(m.y)), x1, s);
                    s = ffma2(make_float2(bf16_lo(m.z), bf16_hi(m.z)), x2, s);
                    acc[r][t] = ffma2(make_float2(bf16_lo(m.w), bf16_hi(m.w)), x3, s);
                }
            }
        }
    }
    // The warp's sums: each step halves the values that a lane holds, then the lanes that hold the
    // same one are added.  A lane ends with value `at`.
    float sum[kN];
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int t = 0; t < kTok; ++t) sum[t * kR + r] = acc[r][t].x + acc[r][t].y;
    int at = 0;
#pragma unroll
    for (int step = 0; step < 5; ++step) {
        const int n = kN >> (step + 1), o = 16 >> step;
        if (n > 0) {
            const bool up = (lane & o) != 0;
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float give = up ? sum[i] : sum[i + n], keep = up ? sum[i + n] : sum[i];
                sum[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
            at += up ? n : 0;
        } else {
            sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], o);
        }
    }
    s_part[warp][at] = sum[0];                     // (lanes with the same value: the same sum)
    if (kWarps > 1) __syncthreads();
    else __syncwarp();
    // one thread an output
    const int i = kWarps > 1 ? (int)threadIdx.x : lane;
    if (i >= feats * kTok) return;
    const int n0 = i / feats * kR + i % feats, t = t0 + i / feats, f = f0 + i % feats;
    if (t >= A.M || f >= A.F) return;
    float y[2];                                    // (gated: the gate and the up)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float s = 0.f;
        const int n = n0 + (h ? kR / 2 : 0);
        if (h == 0 || gated) {
#pragma unroll
            for (int q = 0; q < kWarps; ++q) s += s_part[kWarps > 1 ? q : warp][n];
            if (A.bias) s += load_f32(A.bias + (h ? A.F : 0) + f);
        }
        y[h] = s;
    }
    const size_t o = (size_t)t * A.F + f;
    float out = A.out_f32 ? activate_any<true>(act, y[0]) : activate_any<false>(act, y[0]);
    if (gated) out *= y[1];
    if (A.residual) out += __uint_as_float((uint32_t)A.residual[o] << 16);
    if (A.out_f32) static_cast<float *>(A.out)[o] = out;
    else static_cast<__nv_bfloat16 *>(A.out)[o] = __float2bfloat16_rn(out);
}

// Whether it is faster than the tensor-core kernel: up to two tokens always; three and four up to
// 24 MB of weights (4096 x 2048 6.9 us against 7.6, 4096 x 4096 10.2 against 9.9); five to eight up to
// 12 MB (2048 x 2048 5.6 against 6.0, 4096 x 2048 8.0 against 7.6).  More tokens read the weights once
// for every eight, from L2, and what that reads decides: up to 4 MB (16 tokens 1024 x 1024 4.1
// against 4.4, 24 tokens 5.4 against 4.4; 64 tokens 512 x 512 3.0 against 4.4), or more where the
// tensor cores have one feature block and a long K (64 tokens 8192 x 128 6.8 against 8.5); and the
// rows, whose ends cost as much as short rows do (64 tokens 64 x 1000 3.9 against 3.6).
bool linear_few(const LinearArgs &a, int act) {
    if (a.offsets || a.M > kMostTokens) return false;
    const int times = (a.M + 7) / 8, factor = act == INKATTN_ACT_SWIGLU ? 2 : 1;
    const double rows = (double)a.F * factor, bytes = 2.0 * rows * a.K;
    if (a.M <= 4) return a.M <= 2 || bytes <= 24e6;
    if (rows * times > 6000) return false;
    if (a.M <= 8) return bytes <= 12e6;
    return bytes * times <= 4.2e6 * (rows <= 256 && a.K > 2048 ? a.K / 2048.0 : 1.0);
}

cudaError_t launch_linear_few(const LinearArgs &a, int act, cudaStream_t stream) {
    const int rows = rows_of_group(a.M), feats = act == INKATTN_ACT_SWIGLU ? rows / 2 : rows;
    const int groups = (a.F + feats - 1) / feats;
    const int pieces = a.K / 8;
    auto go = [&](auto kernel, int warps) {
        const int threads = warps * 32 > kFewThreads ? warps * 32 : kFewThreads;
        const int per = threads / (warps * 32);
        return launch_dependent(kernel, dim3((unsigned)((groups + per - 1) / per), (unsigned)((a.M + 7) / 8)), dim3((unsigned)threads), 0, stream, 1, a, act);
    };
    // (sixteen warps a row where there are few rows, so that the SMs have enough requests in flight)
    const int warps = pieces <= 64 ? 1 : groups <= 304 && pieces >= 512 ? 16 : 4;
    auto pick = [&](auto tok) {
        constexpr int kTok = decltype(tok)::value;
        if constexpr (kTok <= 2)
            if (warps == 16) return go(k_linear_few<kTok, 16>, 16);
        return warps == 1 ? go(k_linear_few<kTok, 1>, 1) : go(k_linear_few<kTok, 4>, 4);
    };
    return a.M <= 1 ? pick(std::integral_constant<int, 1>{}) : a.M <= 2 ? pick(std::integral_constant<int, 2>{})
         : a.M <= 4 ? pick(std::integral_constant<int, 4>{}) : pick(std::integral_constant<int, 8>{});
}

}  // namespace inkattn
