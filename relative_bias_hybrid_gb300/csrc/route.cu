// route.cu -- the router's choice of experts, and the weighted sum of the experts' rows.
//
// [SGLang と Miles が Inkling を初日からサポート, §Inkling のモデルアーキテクチャ]: sigmoid
//  scores, the 6 best of 256 routed experts, 2 shared experts that join the normalisation of
//  the weights but not the choice.
//
// Two launches.  k_route_choose: a warp per token holds the token's logits as ordered integer
// keys in registers, each lane knows its own two best, and top_k times the best of the lanes is
// taken (redux.sync on the key, then on the index, so that equal logits go to the lower index).
// A lane looks for its next two only when both are gone.  The next token's logits are requested
// before this one's are used.  k_route_place: a counting sort
// of the (token, choice) pairs by expert, stable in (token, choice) order.  A token takes an
// expert once at most, so the pairs of an expert are a set of tokens, a bitmap: bits are set in
// any order, and the rank of a token among them is a count of bits.  Each block places a chunk of
// the tokens; a pair's row = offset of its expert + pairs of that expert in earlier chunks (each
// block adds up the counts that k_route_choose left per chunk) + bits before its own.  A batch
// that is one chunk needs no counts and no workspace.  (Ranks by match.any and a histogram for
// each warp took 1.6 times as long for one chunk: two passes over the pairs, 32 counts an expert.)
//
// Measured, 6 of 256 + 2: 32768 tokens 27 us (the choice about 19, 475 instructions a token at 0.54
// of the issue rate; 48 warps an SM without the requests ahead took 30), 288 tokens 6.4 us.
#include <type_traits>

#include "common.cuh"
#include "conv4.cuh"
#include "internal.h"

namespace inkattn {

namespace {

constexpr int kChooseThreads = 1024;               // of a chunk; of one chunk alone, fewer
constexpr int kChooseThreadsOne = 256;
// (keys of more than 512 experts want more than the 64 registers of a thread of 1024)
constexpr int choose_threads(int per) { return per > 16 ? kChooseThreads / 2 : kChooseThreads; }
constexpr int kPlaceThreads = 1024;
constexpr int kPlaceTokens = 1024;                 // tokens of a bitmap, a multiple of 32
constexpr int kPlaceOnePairs = 3000;               // pairs of a batch that one block places
constexpr int kChunks = 152;                       // chunks of a larger batch, at most

// Order-preserving integer key of a logit: larger logit, larger key; +0 and -0 alike; NaN as
// -infinity.  Every key is at least 0x007FFFFF; 0 stands for no logit.
__device__ __forceinline__ uint32_t logit_key(float l) {
    const uint32_t u = __float_as_uint(l == l ? l + 0.0f : -INFINITY);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// A lane's two best keys among those it holds that come after (top, e) in the order of choice,
// and their places; equal keys in the order of their places.
struct BestTwo {
    uint32_t k1 = 0, k2 = 0;
    int i1 = 0, i2 = 0;
    __device__ __forceinline__ void add(uint32_t k, int i) {
        const bool first = k > k1, second = k > k2;
        i2 = first ? i1 : second ? i : i2;
        k2 = first ? k1 : second ? k : k2;
        i1 = first ? i : i1;
        k1 = first ? k : k1;
    }
};

}  // namespace

// kPer = logits a lane holds (E <= 32 * kPer); logit e in lane e % 32.  counts: [chunks][E], one
// row written by each block, or NULL for a batch of one chunk.
template <int kPer>
__global__ void __launch_bounds__(choose_threads(kPer), 1)
k_route_choose(const inkattn_route_params p, int chunk_tokens, uint32_t *counts) {
    extern __shared__ uint32_t s_hist[];               // [E], of this block's chunk
    grid_dep_wait();
    grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int width = p.E + p.n_shared, ws = p.top_k + p.n_shared;
    if (counts) {
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) s_hist[e] = 0;
        __syncthreads();
    }
    const int t_lo = blockIdx.x * chunk_tokens, t_hi = min(p.N_tok, t_lo + chunk_tokens);
    const bool sigmoid = p.score == INKATTN_SCORE_SIGMOID;
    const bool is_shared = lane >= p.top_k && lane < ws;
    float next[kPer], next_shared = -INFINITY;
    auto request = [&](int t) {
        const float *row = p.logits + (size_t)t * width;
#pragma unroll
        for (int i = 0; i < kPer; ++i) next[i] = lane + 32 * i < p.E ? load_f32(row + lane + 32 * i) : -INFINITY;
        if (is_shared) next_shared = load_f32(row + p.E + lane - p.top_k);
    };
    if (t_lo + warp < t_hi) request(t_lo + warp);
    for (int t = t_lo + warp; t < t_hi; t += warps) {
        uint32_t key[kPer];
        BestTwo best;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            key[i] = lane + 32 * i < p.E ? logit_key(next[i]) : 0u;
            best.add(key[i], i);
        }
        // lane j < top_k: the j-th choice; the next n_shared lanes: the shared experts
        uint32_t chosen = is_shared ? logit_key(next_shared) : 0u;
        uint32_t id = 0;
        if (t + warps < t_hi) request(t + warps);
        bool two = true;                               // best.k2 is known
        for (int j = 0; j < p.top_k; ++j) {
            const uint32_t top = __reduce_max_sync(0xffffffffu, best.k1);
            const uint32_t mine = best.k1 == top ? (uint32_t)(lane + 32 * best.i1) : 0xffffffffu;
            const uint32_t e = __reduce_min_sync(0xffffffffu, mine);
            const bool taken = mine == e;
            if (lane == j) {
                chosen = top;
                id = e;
            }
            if (__any_sync(0xffffffffu, taken && !two)) {
                BestTwo rest;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const bool after = key[i] < top || (key[i] == top && (uint32_t)(lane + 32 * i) > e);
                    rest.add(after ? key[i] : 0u, i);
                }
                if (taken) {
                    best = rest;
                    two = true;
                }
            } else if (taken) {
                best.k1 = best.k2;
                best.i1 = best.i2;
                two = false;
            }
        }
        // Scores up to a factor common to the token, so that they do not all vanish: softmax
        // exp(l - m) with m the largest logit; sigmoid exp(l - m) / (1 + exp(l)) with m the largest
        // logit or 0, whichever is less.  For m = 0 that is the sigmoid, from one exponential:
        // with e = exp(-|l|), 1 / (1 + e) for a positive l and e / (1 + e) for others.
        const float l = key_logit(chosen), top_l = key_logit(__reduce_max_sync(0xffffffffu, chosen));
        float s;
        if (sigmoid && top_l >= 0.f) {
            const float e = expf(-fabsf(l));
            s = __fdividef(l > 0.f ? 1.f : e, 1.f + e);
        } else {
            s = l == top_l ? 1.f : expf(l - top_l);                          // (equal infinities too)
            if (sigmoid) s = __fdividef(s, 1.f + expf(l));
        }
        if (lane >= ws || l == -INFINITY) s = 0.f;
        float sum = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane < ws) p.weights[(size_t)t * ws + lane] = sum > 0.f ? p.scale * __fdividef(s, sum) : 0.f;
        if (lane < p.top_k) {
            p.topk_ids[(size_t)t * p.top_k + lane] = (int32_t)id;
            if (counts) atomicAdd(&s_hist[id], 1u);    // (integers: the order does not show)
        }
    }
    if (counts) {
        __syncthreads();
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) counts[(size_t)blockIdx.x * p.E + e] = s_hist[e];
    }
}

// One block per chunk.  Shared memory: base[E] (row of the expert's next pair), scratch[2
// kPlaceThreads], bits[words][E], before[words][E] (16 bits: bits in earlier words).
__global__ void __launch_bounds__(kPlaceThreads)
k_route_place(const inkattn_route_params p, int chunk_tokens, int words, const uint32_t *counts) {
    extern __shared__ uint32_t sm[];
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int E = p.E, k = p.top_k;
    const uint32_t all = (uint32_t)p.N_tok * (uint32_t)k;
    uint32_t *base = sm, *scratch = sm + E, *bits = scratch + 2 * kPlaceThreads;
    uint16_t *earlier = reinterpret_cast<uint16_t *>(bits + words * E);
    const int t_lo = (int)min((long long)blockIdx.x * chunk_tokens, (long long)p.N_tok);
    const int t_hi = min(p.N_tok - t_lo, chunk_tokens) + t_lo;

    // base and expert_offsets from the totals of the experts; `before`: pairs of earlier chunks
    auto start_rows = [&](uint32_t total, uint32_t before) {
        uint32_t v = tid < E ? total : 0u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t n = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += n;
        }
        if (lane == 31) scratch[warp] = v;
        __syncthreads();
        uint32_t s = lane < warp ? scratch[lane] : 0u;         // (32 warps: the totals of the earlier ones)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (tid < E) {
            const uint32_t incl = v + s;
            base[tid] = incl - total + before;
            if (blockIdx.x == 0) {
                p.expert_offsets[tid + 1] = (int32_t)incl;
                if (tid == 0) p.expert_offsets[0] = 0;
            }
        }
    };
    if (counts) {
        // several threads an expert, each over a part of the chunks
        const int parts = kPlaceThreads / E, e = tid % E, part = tid / E, chunks = gridDim.x;
        uint32_t total = 0, before = 0;
        if (part < parts) {
            for (int c0 = part; c0 < chunks; c0 += 8 * parts) {
                uint32_t n[8];                         // requested together
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int c = c0 + q * parts;
                    n[q] = c < chunks ? load_u32(counts + (size_t)c * E + e) : 0u;
                }
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    total += n[q];
                    before += c0 + q * parts < (int)blockIdx.x ? n[q] : 0u;
                }
            }
            scratch[2 * tid] = total;
            scratch[2 * tid + 1] = before;
        }
        __syncthreads();
        total = before = 0;
        if (tid < E) {
            for (int q = 0; q < parts; ++q) {
                total += scratch[2 * (q * E + tid)];
                before += scratch[2 * (q * E + tid) + 1];
            }
        }
        __syncthreads();
        start_rows(total, before);
    }
    int t0 = t_lo;
    do {                                               // (once at least: an empty batch has offsets too)
        const int t1 = min(t_hi, t0 + 32 * words);
        for (int i = tid; i < words * E; i += kPlaceThreads) bits[i] = 0;
        __syncthreads();
        const int pairs = (t1 - t0) * k;
        const int32_t *ids = p.topk_ids + (size_t)t0 * k;
        for (int q = tid; q < pairs; q += kPlaceThreads) {
            const int t = q / k;
            atomicOr(&bits[(t >> 5) * E + ids[q]], 1u << (t & 31));
        }
        __syncthreads();
        uint32_t run = 0;
        if (tid < E) {
#pragma unroll 4
            for (int w = 0; w < words; ++w) {
                earlier[w * E + tid] = (uint16_t)run;
                run += __popc(bits[w * E + tid]);
            }
        }
        if (!counts) start_rows(run, 0);
        __syncthreads();
        for (int q = tid; q < pairs; q += kPlaceThreads) {
            const int t = q / k, e = ids[q], w = t >> 5;
            const uint32_t row = base[e] + earlier[w * E + e] + __popc(bits[w * E + e] & ((1u << (t & 31)) - 1u));
            if (row < all) p.row_token[row] = t0 + t;  // (always, unless another call wrote the counts)
            p.token_rows[(size_t)t0 * k + q] = (int32_t)row;
        }
        t0 += 32 * words;
        if (t0 < t_hi) {
            __syncthreads();
            if (tid < E) base[tid] += run;
            __syncthreads();
        }
    } while (t0 < t_hi);
}

// One block places few pairs sooner than many blocks do, which need the counts first: 500 tokens
// with 6 choices 7.7 us against 8.2, 1000 tokens 10.4 against 8.4 (and 64 experts, 4 choices 7.7 against 6.3).
static bool one_chunk(const inkattn_route_params &p) {
    return p.N_tok <= kPlaceTokens && p.N_tok * p.top_k <= kPlaceOnePairs;
}
static int chunk_tokens(const inkattn_route_params &p) {
    const int t = (p.N_tok + kChunks - 1) / kChunks;
    return t < 32 ? 32 : t;
}

size_t route_workspace_bytes(const inkattn_route_params &p) {
    if (one_chunk(p)) return 0;
    const int t = chunk_tokens(p);
    return (size_t)((p.N_tok + t - 1) / t) * p.E * 4;
}

cudaError_t launch_route(const inkattn_route_params &p, uint32_t *ws, cudaStream_t stream) {
    const bool one = one_chunk(p);
    // the choice of a small batch: a token per warp
    const int choose_tokens = one ? kChooseThreadsOne / 32 : chunk_tokens(p);
    const int place_tokens = one ? (p.N_tok > 0 ? p.N_tok : 1) : chunk_tokens(p);
    uint32_t *counts = one ? nullptr : ws;
    cudaError_t err = cudaSuccess;
    if (p.N_tok > 0) {
        const dim3 grid((unsigned)((p.N_tok + choose_tokens - 1) / choose_tokens));
        const size_t smem = one ? 0 : (size_t)p.E * 4;
        auto go = [&](auto kernel, int per) {
            const int threads = one ? kChooseThreadsOne : choose_threads(per);
            return launch_dependent(kernel, grid, dim3((unsigned)threads), smem, stream, 1, p, choose_tokens, counts);
        };
        err = p.E <= 64 ? go(k_route_choose<2>, 2) : p.E <= 128 ? go(k_route_choose<4>, 4) : p.E <= 256
            ? go(k_route_choose<8>, 8) : p.E <= 384 ? go(k_route_choose<12>, 12) : p.E <= 512 ? go(k_route_choose<16>, 16)
            : go(k_route_choose<32>, 32);
        if (err != cudaSuccess) return err;
    }
    const int words = ((place_tokens < kPlaceTokens ? place_tokens : kPlaceTokens) + 31) / 32;
    auto smem_of = [](int E, int w) { return (size_t)E * 4 + 2 * kPlaceThreads * 4 + (size_t)w * E * 6; };
    err = cudaFuncSetAttribute(k_route_place, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)smem_of(INKATTN_MAX_EXPERTS, kPlaceTokens / 32));
    if (err != cudaSuccess) return err;
    const dim3 grid((unsigned)(one ? 1 : (p.N_tok + place_tokens - 1) / place_tokens));
    return launch_dependent(k_route_place, grid, dim3(kPlaceThreads), smem_of(p.E, words), stream, 1, p, place_tokens, words,
                            static_cast<const uint32_t *>(counts));
}

// ---------------------------------------------------------------- the weighted sum
// HBM-bound: top_k + n_shared rows read and one written per token.  A thread owns 8 features
// (a 16-byte piece of every row) of one token, or, where a token has few rows, of two, four or
// eight, and requests up to eight pieces before it uses the first; the sum is taken in fp32 in the
// order of the choices.  Narrow rows: several tokens a block.  Measured: 8192 tokens x 8 rows of
// 8192 in 182 us, 6.6 TB/s (98% of the copy rate); 288 tokens in 9.2 us; 8192 tokens with one row of
// 8192 49 us (94 with one token a thread), with ten of 64 4.7 us (12 with one token a block).

namespace {
constexpr int kSumThreads = 128;
constexpr int kSumRows = 8;                        // pieces requested at once
constexpr int kSumResident = 152 * 2048 / kSumThreads;   // blocks that run at once
}  // namespace

// A thread sums kRows rows of kTokens tokens at a time.  kWide: the block is one token's (the same
// in every thread, so that its weights and rows are read once a warp: 182 us where 192 otherwise),
// else 1 << shift threads are; chunks: blocks of a row's pieces.
template <bool kWide, int kRows, int kTokens>
__global__ void __launch_bounds__(kSumThreads)
k_expert_combine(const inkattn_expert_combine_params p, int shift, int chunks) {
    static_assert(kRows * kTokens <= kSumRows, "pieces requested at once");
    grid_dep_wait();
    grid_dep_launch();
    const int G = p.F >> 3;                            // 16-byte pieces of a row
    const int tokens = kWide ? 1 : kSumThreads >> shift;   // side by side in the block
    const int group = (int)blockIdx.x / chunks, chunk = (int)blockIdx.x - group * chunks;
    const int g = kWide ? chunk * kSumThreads + (int)threadIdx.x : (int)threadIdx.x & ((1 << shift) - 1);
    const long long t0 = (long long)group * (tokens * kTokens) + (kWide ? 0 : (int)threadIdx.x >> shift);
    if (g >= G || t0 >= p.N_tok) return;
    const int rows = p.top_k + p.n_shared;
    const uint4 *y = reinterpret_cast<const uint4 *>(p.y), *sh = reinterpret_cast<const uint4 *>(p.shared);
    float acc[kTokens][8] = {};
    for (int j0 = 0; j0 < rows; j0 += kRows) {
        uint4 v[kTokens][kRows];
        float c[kTokens][kRows];
#pragma unroll
        for (int n = 0; n < kTokens; ++n) {
            const long long t = t0 + n * tokens;
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int j = j0 + i;
                v[n][i] = make_uint4(0, 0, 0, 0);
                c[n][i] = 0.f;
                if (j >= rows || (kTokens > 1 && t >= p.N_tok)) continue;
                if (j < p.top_k) {
                    const int r = load_i32(p.token_rows + t * p.top_k + j);
                    if (r >= 0 && r < p.M) {
                        c[n][i] = load_f32(p.weights + t * rows + j);
                        v[n][i] = __ldcs(y + (size_t)r * G + g);
                    } else if (r != -1 && g == 0) {
                        set_status(p.dev_status, INKATTN_ERR_DEVICE_BOUNDS);
                    }
                } else {
                    c[n][i] = load_f32(p.weights + t * rows + j);
                    v[n][i] = __ldcs(sh + ((size_t)(j - p.top_k) * p.N_tok + t) * G + g);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < kTokens; ++n)
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                float x[8];
                unpack8(v[n][i], x);
#pragma unroll
                for (int m = 0; m < 8; ++m) acc[n][m] = fmaf(c[n][i], x[m], acc[n][m]);
            }
    }
#pragma unroll
    for (int n = 0; n < kTokens; ++n) {
        const long long t = t0 + n * tokens;
        if (kTokens == 1 || t < p.N_tok) reinterpret_cast<uint4 *>(p.out)[t * G + g] = pack8(acc[n]);
    }
}

cudaError_t launch_expert_combine(const inkattn_expert_combine_params &p, cudaStream_t stream) {
    const int G = p.F / 8, rows = p.top_k + p.n_shared;
    int shift = 0;
    while ((1 << shift) < G && (1 << shift) < kSumThreads) ++shift;
    const int chunks = (G + (1 << shift) - 1) >> shift, tokens = kSumThreads >> shift;
    auto blocks = [&](int n) { return ((long long)p.N_tok + tokens * n - 1) / (tokens * n) * chunks; };
    auto go = [&](auto kernel, int n) {
        return launch_dependent(kernel, dim3((unsigned)blocks(n)), dim3(kSumThreads), 0, stream, 1, p, shift, chunks);
    };
    // Several tokens a thread only for more blocks than run at once: with fewer, more threads
    // are more requests in flight.
    auto pick = [&](auto wide) {
        constexpr bool kWide = decltype(wide)::value;
        if (rows > 4 || blocks(1) <= kSumResident) return go(k_expert_combine<kWide, 8, 1>, 1);
        if (rows > 2) return go(k_expert_combine<kWide, 4, 2>, 2);
        if (rows > 1) return go(k_expert_combine<kWide, 2, 4>, 4);
        return go(k_expert_combine<kWide, 1, 8>, 8);
    };
    return tokens == 1 ? pick(std::true_type{}) : pick(std::false_type{});
}

}  // namespace inkattn
