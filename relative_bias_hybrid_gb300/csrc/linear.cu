// linear.cu -- linear layers and the experts' grouped products on the 5th-generation tensor
// cores (TMA + tcgen05/TMEM): bias, activation and residual in the GEMM's epilogue.
//
// [vLLM hỗ trợ TML Inkling ..., §TP sharding nhận biết sconv]: the output projection in front
//  of the attention-output conv.
// [SGLang と Miles が Inkling を初日からサポート, §Inkling のモデルアーキテクチャ]: the MoE's
//  routed and shared experts.
//
// out[i][f] = act( sum_k x[s_i][k] w[e][f][k] + bias[e][f] ) + residual[i][f] over the rows i of
// each expert e; a linear layer is the case of one expert that owns every row (of few tokens:
// linear_few.cu).
//
// Orientation.  The weight rows are the MMA's M side and the tokens its N side: a work item is
// 256 weight rows times up to 256 tokens, computed by the two CTAs of a pair as one
// M = 256 tile (tcgen05 cta_group::2), and N is the item's own token count rounded up to 32.
// A decode batch or an expert with few rows thus pays for the rows it has (N = 32 takes an
// eighth of the tensor time of N = 256), while the weights, which bound such a call, stream
// through at full width.  Each CTA holds its own 128 weight rows and half of the tokens.
//
// The rows of a token tile are one box of x, as many rows as the tile has (a tensor map for
// each box height), or, with row indices, are gathered by four warps of their own with 16-byte
// cp.async: the copy of x in expert order is never written.  (TMA's gather of four rows was
// measured first: a K = 64 step of 128 rows took about 1800 cycles, 3.5 times its MMAs.)
//
// SWIGLU: the CTA's 128 weight rows are 64 gate rows and the 64 up rows of the same features, one
// box; the two warps that hold a feature's gate and up exchange half of the tokens through shared
// memory.  (16 gate rows and 16 up rows in turn, a shuffle apart in one warp, were measured first:
// four boxes a stage made the copies the bound, 0.78 ms where one box takes 0.57 for the same
// products.)
//
// One CTA per SM, 11 warps (16 with row indices):
//   warps 0, 10 producers, a lane of each: copies of the weight rows and the token rows into a
//               ring of stages of K = 64, as many as fit 192 KB, the two taking turns: a stage
//               costs its producer about 400 cycles (the wait, the barrier, two copies), which a
//               single one made the bound of every tile below N = 256
//   warp 1      even CTA: MMA issuer, K = 16 steps into one of two TMEM accumulators (2 x 256
//               columns), so that an item's epilogue overlaps the next item's MMAs
//   warps 11-14 only with row indices: the gather; warp 15 hands its stages to the MMA warp
//   warps 2-9   epilogue: a warp owns 32 TMEM lanes (weight rows) and every second block of 32
//               columns (tokens); bias and activation per lane, and each value leaves from the lane
//               that has it, a token's 32 features together.  (Turned through shared memory first, so
//               that they left as 16-byte pieces: 31 us as well for 8192 x 512 x 4096, and 50 where this
//               takes 46 with a residual.  What the stores do cost is a predicate each: blocks
//               whose tokens are all there go without, 53 -> 29 us for 8192 x 512 x 4095.)
// Both CTAs' copies of a stage complete on the even CTA's barrier, and the pair's commits
// release it in both, as in the qkvr kernel.
//
// fp32 outputs (kFine).  The tensor cores add each K = 16 step to the accumulator without rounding
// to nearest; over K = 8192 the error grows to about 1e-5 of the result, nothing next to a bf16
// rounding but much for an fp32 one.  An fp32 output is therefore summed in parts of K = 512,
// which the epilogue warps add up in TMEM, rounding to nearest (K = 1000: 4.7e-7 of the result
// instead of 9.8e-7, and the same at K = 8192).  The two accumulators and the sums share the 512
// TMEM columns, so the tiles have 160 tokens at most: 8192 x 8192 x 8192 takes 0.64 ms instead of
// 0.57 (0.72 against 0.64 under the power cap).
//
// Few items (a decode batch): the K range is split over the S pairs of one cluster.  Each CTA
// writes its fp32 partial tile, a share of the tokens to each pair, into the other CTAs' shared
// memory (the rings, idle by then), and each adds the S partials of its share in order: no
// workspace, no atomics, one launch.  (Reading the partials from the other CTAs instead took
// 11000 cycles for 256 tokens and S = 4: 12 bytes a cycle.)
//
// Measured (back to back on one GB300): 8192 x 8192 x 8192 0.57 ms, 1920 TFLOP/s in a burst with
// the tensor pipe 89.5% active, 0.64 to 0.67 (1650 to 1720) under the power cap; 4 x 8192 x 8192 23.3
// us, the weights at 7.2 TB/s for 18.5 of them; 288 x 8192 x 8192 33.5 us, 37 with a residual (two
// tiles: 26 KB a K step at the 64 bytes a cycle into an SM); 256 experts 8192 -> 2 x 1024 for 1728
// gathered rows 1.01 to 1.07 ms, 8.0 to 8.5 TB/s of weights; 64 experts 4096 -> 2 x 2048 for 49152
// gathered rows 1.03 ms in a burst (1600 TFLOP/s, tensor pipe 75%; 0.98 ms on contiguous rows), 1.14
// to 1.19 under the power cap (1390 to 1450).
#include <climits>
#include <cmath>
#include <type_traits>

#include "activation.cuh"
#include "common.cuh"
#include "device_table.h"
#include "internal.h"
#include "tcgen05.cuh"
#include "cta_pair.cuh"

namespace inkattn {

namespace {

constexpr int kRowsA = 128;                       // weight rows of a CTA
constexpr int kMaxN = 256;                        // tokens of an item
constexpr int kKStep = 64;                        // K per ring stage (one 128-byte row)
constexpr int kABytes = kRowsA * 128;             // 16 KB
constexpr int kRingBytes = 192 * 1024;
constexpr int kMaxStages = 12;
constexpr int kMaxSplits = 4;                     // pairs of a cluster (eight CTAs)
constexpr int kThreads = 352;                     // without a gather
constexpr int kGatherWarps = 4, kGatherTeam = 64;  // threads that gather a stage together
constexpr int kMaxThreads = kThreads + kGatherWarps * 32 + 32;
constexpr int kEpiThreads = 256;
constexpr int kWarpProducer = 0, kWarpMma = 1, kWarpEpi = 2, kWarpProducer2 = 10, kWarpGather = 11,
              kWarpRelay = 15;
constexpr int kStgPitch = 32;                     // SWIGLU: floats of a row of the exchange, 32 features
constexpr int kStgBytes = 16 * kStgPitch * 4;     // 16 tokens, one buffer per epilogue warp
constexpr int kFineSteps = 8, kFineN = 160;       // fp32 outputs: K steps of a part, tokens of a tile
constexpr int kSetupBar = 5;                      // named barrier (1 to 4: SWIGLU's exchanges)
constexpr int kRaster = 8;                        // feature blocks per raster group

constexpr int kOffStg = kRingBytes;
constexpr int kNoteBytes = 16;                    // the odd CTA's note that a gathered stage is complete
constexpr int kOffNote = kOffStg + 8 * kStgBytes; // where it lands, and behind it what is sent
constexpr int kOffTiles = kOffNote + 2 * kNoteBytes;                   // int tile prefix [E + 1]
constexpr int kOffStart = kOffTiles + (INKATTN_MAX_EXPERTS + 1) * 4;   // int first row [E + 1]
constexpr int kOffPer = kOffStart + (INKATTN_MAX_EXPERTS + 1) * 4;     // int rows of a tile [E]
constexpr int kOffBar = (kOffPer + INKATTN_MAX_EXPERTS * 4 + 7) / 8 * 8;
enum Bar {
    B_FULL = 0,
    B_EMPTY = B_FULL + kMaxStages,
    B_GATHER = B_EMPTY + kMaxStages,
    B_ACC_FULL = B_GATHER + kMaxStages,
    B_ACC_EMPTY = B_ACC_FULL + 2,
    B_DRAIN = B_ACC_EMPTY + 2,
    B_COUNT = B_DRAIN + 1
};
constexpr int kSmem = kOffBar + B_COUNT * 8 + 16;
static_assert(kMaxN / 32 <= sizeof(LinearMaps::x) / sizeof(CUtensorMap), "a map for each box height");
static_assert(kSmem <= 232448, "dynamic shared memory above the 227 KB a CTA may use");
static_assert(kMaxN * kRowsA * 4 <= kRingBytes, "a split's partial tile lies in the ring");

struct Item {
    int e, row0, nt, n, fb;      // expert, first row, rows, MMA N (rows rounded up to 32), feature block
};

__device__ __forceinline__ void store_bf16(inkattn_bf16 *p, float v) {
    *reinterpret_cast<__nv_bfloat16 *>(p) = __float2bfloat16_rn(v);
}
__device__ __forceinline__ float load_bf16(const inkattn_bf16 *p) { return __uint_as_float((uint32_t)*p << 16); }

// 16 bytes global -> shared without a register stop; all zeros where `live` is false
__device__ __forceinline__ void cp_async16(uint32_t dst, uint64_t src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void *p) {
    asm volatile("prefetch.global.L2 [%0];" :: "l"(reinterpret_cast<uint64_t>(p)));
}
// arrives on the mbarrier once this thread's earlier cp.async have landed
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// bar.sync over n threads, and the same reducing a predicate with AND
__device__ __forceinline__ void named_sync(int id, int n) { asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ bool named_all(int id, int n, bool v) {
    int r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbar.red.and.pred q, %2, %3, p;\n\t"
                 "selp.s32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"((int)v), "r"(id), "r"(n) : "memory");
    return r != 0;
}

// A position in the ring: stage and how often the ring has been passed (its low bit: the parity).
struct RingPos {
    int s = 0;
    uint32_t lap = 0;
    __device__ __forceinline__ void next(int stages, int by = 1) {
        s += by;
        if (s >= stages) {
            s -= stages;
            ++lap;
        }
    }
};

__device__ __forceinline__ void st_shared_cluster(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" :: "r"(addr), "r"(v) : "memory");
}

// The token tiles of the experts, in shared memory: the prefix of their counts, each expert's
// first row (and the last one's end), and the rows of a tile.
struct Tiles {
    int *prefix, *start, *per;
    int most;                                          // units of 32 rows of a tile
    // An expert's tiles: of near-equal size, a multiple of 32 rows.
    __device__ __forceinline__ int enter(int e, int first, int rows) const {
        const int units = (int)(((uint32_t)rows + 31) >> 5);
        int tiles = units > 0, each = units;
        if (units > most) {
            tiles = (units - 1) / most + 1;
            each = (units - 1) / tiles + 1;
        }
        start[e] = first;
        per[e] = each * 32;
        return tiles;
    }
};

// The tiles of more than 32 experts from their offsets, by warps w = 0 .. 7 (by one, 32 experts at a
// time, each took 0.6 us: a token for 256 experts 10.3 us where this takes 6.3).  A function of its
// own, of rolled loops: it runs once, from a cold instruction cache, and beside the code that follows
// it slowed everything down (linear layers by 0.4 us, eight experts a lane unrolled all by 1.3).
__device__ __noinline__ void setup_experts(Tiles t, const int32_t *offsets, int E, int M, int w, int lane, int *scan,
                                           int32_t *dev_status) {
    constexpr int kWarps = kEpiThreads / 32;
    int carry = 0;
    bool ok = true;
#pragma unroll 1
    for (int e0 = 0, round = 0; e0 < E; e0 += kEpiThreads, round ^= kWarps) {
        const int e = e0 + w * 32 + lane;
        int v = 0;                                     // tiles, then tiles up to this expert
        if (e < E) {
            const int first = offsets[e], end = offsets[e + 1];
            const bool possible = first >= 0 && end >= first && end <= M;
            ok = ok && possible;
            v = t.enter(e, first, possible ? end - first : 0);
            if (e == E - 1) t.start[E] = end;
        }
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += n;
        }
        if (lane == 31) scan[round + w] = v;           // (two halves in turn: the next round's writes)
        ok = named_all(kSetupBar, kEpiThreads, ok);
        const int of = lane < kWarps ? scan[round + lane] : 0;
        v += carry + __reduce_add_sync(0xffffffffu, lane < w ? of : 0);
        carry += __reduce_add_sync(0xffffffffu, of);
        if (e < E) t.prefix[e + 1] = v;
    }
    if (!ok) named_sync(kSetupBar, kEpiThreads);       // (nobody writes after the thread below)
    if (w > 0 || lane > 0) return;
    t.prefix[0] = 0;
    if (ok) return;
    // Some offsets are impossible: one expert after another.
    set_status(dev_status, INKATTN_ERR_DEVICE_BOUNDS);
    int reached = 0, before = 0;
#pragma unroll 1
    for (int e = 0; e < E; ++e) {
        const int first = offsets[e], end = offsets[e + 1];
        const bool possible = first >= 0 && end >= first && end <= M;
        before += t.enter(e, first, possible && first >= reached ? end - first : 0);
        t.prefix[e + 1] = before;
        if (possible) reached = max(reached, end);
    }
}

}  // namespace

// kFine: fp32 output, summed in parts.  kResid: with a residual, and then without row indices (the
// registers of the gather's threads hold residual values).
template <int kAct, bool kFine, bool kResid>
__global__ void __launch_bounds__(kResid ? kThreads : kMaxThreads, 1)
k_linear(const LinearArgs A, const __grid_constant__ LinearMaps maps) {
    constexpr bool kGated = kAct == INKATTN_ACT_SWIGLU;
    constexpr int kFeat = kGated ? 64 : 128;           // output features of a CTA
    extern __shared__ __align__(1024) unsigned char smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t crank = cluster_ctarank();
    const int half = (int)(crank & 1u);                // CTA of the pair
    const uint32_t even = crank & ~1u;                 // the pair's even CTA
    const int split = (int)(crank >> 1);               // which part of K this pair takes
    const int cid = (int)blockIdx.x / (2 * A.splits), nclusters = (int)gridDim.x / (2 * A.splits);
    const uint32_t s_base = smem_u32(smem);
    if ((s_base & 1023u) != 0u) {                      // the same in every CTA
        grid_dep_wait();
        if (threadIdx.x == 0) set_status(A.dev_status, INKATTN_ERR_DEVICE_BOUNDS);
        return;
    }
    auto bar = [&](int i) { return s_base + kOffBar + 8u * (uint32_t)i; };
    int *s_tiles = reinterpret_cast<int *>(smem + kOffTiles);
    int *s_start = reinterpret_cast<int *>(smem + kOffStart);
    int *s_per = reinterpret_cast<int *>(smem + kOffPer);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kOffBar + B_COUNT * 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffBar + B_COUNT * 8 + 4);
    // a stage of the ring: completed by copies or by a commit, which carry their own ordering
    auto pwait = [&](uint32_t addr, uint32_t parity) -> bool {
        const bool r = mbar_wait_short<200>(addr, parity, A.dev_status, abort_flag, A.wait_ns);
        return __all_sync(0xffffffffu, r);
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < A.stages; ++s) {
            mbar_init(bar(B_FULL + s), A.row_token ? 2 : 1);   // (the even CTA's: both CTAs' copies, its relay)
            mbar_init(bar(B_GATHER + s), kGatherTeam);
            mbar_init(bar(B_EMPTY + s), 1);            // released by the pair's MMAs
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(B_ACC_FULL + s), 1);
            mbar_init(bar(B_ACC_EMPTY + s), 16);       // every epilogue warp of both CTAs
        }
        mbar_init(bar(B_DRAIN), 1);
        *abort_flag = 0;
        *reinterpret_cast<uint4 *>(smem + kOffNote + kNoteBytes) = make_uint4(0, 0, 0, 0);
        fence_mbar_init();
    }
    if (warp == kWarpMma) {                            // with the peer CTA's MMA warp
        tc::tmem_alloc_pair(smem_u32(tmem_slot), 512);
        tc::tmem_relinquish_pair();
    }
    // Everything up to here and, for a linear layer, the rest of the setup needs no global memory
    // and runs while the kernel before this one on the stream finishes; each role waits for that
    // kernel before it reads or writes global memory, and before its first wait with a limit.
    // First row of every expert, rows of its token tiles, and the prefix of the tiles: s_tiles[e] =
    // tiles of experts 0 .. e-1.  An expert that reaches back into the rows of an earlier one is refused
    // like one with impossible offsets: the accepted ones hold M rows together at most, so that the
    // items stay within what the launch was sized for.
    const Tiles tiles = {s_tiles, s_start, s_per, A.tile_n >> 5};
    if (A.E > 32) {
        if (warp >= kWarpEpi && warp < kWarpEpi + kEpiThreads / 32) {
            grid_dep_wait();
            setup_experts(tiles, A.offsets, A.E, A.M, warp - kWarpEpi, lane, reinterpret_cast<int *>(smem + kOffStg),
                          A.dev_status);
        }
    } else if (warp == kWarpEpi) {
        if (A.offsets) grid_dep_wait();
        const bool there = lane < A.E;
        const int start = there && A.offsets ? A.offsets[lane] : 0;
        const int end = there ? A.offsets ? A.offsets[lane + 1] : A.M : 0;
        bool valid = start >= 0 && end >= start && end <= A.M;
        int most = valid ? end : 0;                    // largest end up to this lane, then before it
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, most, o);
            if (lane >= o) most = max(most, n);
        }
        most = __shfl_up_sync(0xffffffffu, most, 1);
        valid = valid && there && start >= (lane ? most : 0);
        int v = there ? tiles.enter(lane, start, valid ? end - start : 0) : 0;
        if (there && !valid) set_status(A.dev_status, INKATTN_ERR_DEVICE_BOUNDS);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += n;
        }
        if (there) s_tiles[lane + 1] = v;
        if (lane == A.E - 1) s_start[A.E] = end;
        if (lane == 0) s_tiles[0] = 0;
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    cluster_sync();                                    // the peers' barriers exist
    const uint32_t tmem = *tmem_slot;

    const int n_items = s_tiles[A.E] * A.n_fblocks;    // (the host checked that it fits)
    const int nk = (A.K + kKStep - 1) / kKStep;
    const int k_lo = (int)((long long)nk * split / A.splits), k_hi = (int)((long long)nk * (split + 1) / A.splits);
    // the accumulations of an item, one after another in the two TMEM buffers
    const int part = kFine ? kFineSteps : k_hi - k_lo, parts = kFine ? (k_hi - k_lo + part - 1) / part : 1;
    const int my_items = cid < n_items ? (n_items - cid + nclusters - 1) / nclusters : 0;
    constexpr int kAccCols = kFine ? kFineN : kMaxN;           // TMEM columns of an accumulator
    const uint32_t t_sums = tmem + 2 * kFineN;                 // kFine: the sums of the parts so far
    auto item = [&](int w) {
        // (integer divisions are some hundred cycles together: as few as there can be)
        Item it;
        int lo = 0, hi = A.E;                          // s_tiles[lo] <= t < s_tiles[hi]
        if (hi > 1) {
            const int t = w / A.n_fblocks;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_tiles[mid] <= t) lo = mid;
                else hi = mid;
            }
        }
        it.e = lo;
        // the expert's items: groups of kRaster feature blocks, inside a group the token tiles
        // one after another, so that the group's weights stay in L2 while they stream past
        const int mt = s_tiles[lo + 1] - s_tiles[lo];
        const int rem = w - s_tiles[lo] * A.n_fblocks;
        const int grp = mt == 1 ? rem / kRaster : rem / (kRaster * mt), in = rem - grp * kRaster * mt;
        const int gsz = min(kRaster, A.n_fblocks - grp * kRaster);
        const int m = mt == 1 ? 0 : gsz == kRaster ? in / kRaster : in / gsz;
        it.fb = grp * kRaster + (in - m * gsz);
        const int rows = s_start[lo + 1] - s_start[lo], per = s_per[lo];
        it.row0 = s_start[lo] + m * per;
        it.nt = min(per, rows - m * per);
        it.n = (it.nt + 31) & ~31;
        return it;
    };

    // a split's cluster has one item at most (worked out here, off the path behind the products)
    const Item only = A.splits > 1 && cid < n_items ? item(cid) : Item{};

    if (warp == kWarpProducer || warp == kWarpProducer2) {
        // ================================ producers ================================
        if (lane == 0) {
            const int turn = warp == kWarpProducer ? 0 : 1;
            if (turn == 0) {
                if (!A.row_token) tma_prefetch_desc(&maps.x[0]);
                tma_prefetch_desc(&maps.w);
            }
            grid_dep_wait();
            if (turn == 0) grid_dep_launch();
            const uint32_t full = mapa_shared(bar(B_FULL), even);
            RingPos at;
            at.s = turn;
            int first = turn, last = -1;               // of an item's loads, the first of this warp's; its newest load
            int base = 0;                              // loads of the items before
            bool ok = true;
            for (int w = cid; w < n_items && ok; w += nclusters) {
                const Item it = item(w);
                const int hn = it.n >> 1;              // tokens of a CTA's half of the tile
                const uint32_t bytes = 2 * kABytes + (A.row_token ? kNoteBytes : 2u * (uint32_t)hn * 128u);
                const CUtensorMap *xm = &maps.x[(hn >> 4) - 1];
                const int wrow = (it.fb * 2 + half) * kFeat, xrow = it.row0 + half * hn;
                int k = k_lo + first;
                for (; k < k_hi; k += 2, at.next(A.stages, 2)) {
                    if (at.lap > 0 && !mbar_wait_short<200>(bar(B_EMPTY + at.s), (at.lap - 1) & 1, A.dev_status, abort_flag,
                                                         A.wait_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = s_base + (uint32_t)(at.s * A.stage_bytes), fb = full + 8u * (uint32_t)at.s;
                    if (half == 0) mbar_arrive_expect_tx(bar(B_FULL + at.s), bytes);
                    if (kGated) tma_load_4d_pair(dst, &maps.w, k * kKStep, wrow, 0, it.e, fb);
                    else tma_load_3d_pair(dst, &maps.w, k * kKStep, wrow, it.e, fb);
                    if (!A.row_token) tma_load_2d_pair(dst + kABytes, xm, k * kKStep, xrow, fb);
                    last = base + k - k_lo;
                }
                first = k - k_hi;
                base += k_hi - k_lo;
            }
            // nothing may still be landing in shared memory when the pair tears down: the even
            // CTA waits for the last lap of both CTAs' copies (see qkvr.cu), for the loads whose stage
            // the other producer's newest load cannot have taken over
            if (half == 0)
                for (int l = last; l >= 0 && l > last + 1 - A.stages; l -= 2)
                    (void)mbar_wait_short<200>(bar(B_FULL + l % A.stages), (uint32_t)(l / A.stages) & 1u, A.dev_status,
                                               nullptr, A.wait_ns);
        }
        __syncwarp();
    } else if (warp == kWarpRelay) {
        // ================================ relay ================================
        // The gathered rows were written through the generic proxy and the MMAs read through the
        // async one: a fence between the two, by a warp that has no copies of its own in flight,
        // once a stage's rows have landed.  The odd CTA then tells the even one by a 16-byte bulk
        // copy, an async operation that the fence orders behind the rows and whose bytes complete
        // on the even CTA's barrier.  (A remote arrival with release at cluster scope stalled the
        // warp for about 1 us a stage: 2.7 ms where this takes 1.1.)
        grid_dep_wait();
        RingPos at;
        bool ok = true;
        for (int w = cid; w < n_items && ok; w += nclusters)
            for (int k = k_lo; k < k_hi; ++k, at.next(A.stages)) {
                ok = pwait(bar(B_GATHER + at.s), at.lap & 1);
                if (!ok) break;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (half == 0) mbar_arrive(bar(B_FULL + at.s));
                    else bulk_copy_pair(mapa_shared(s_base + kOffNote, even), s_base + kOffNote + kNoteBytes, kNoteBytes,
                                        mapa_shared(bar(B_FULL + at.s), even));
                }
            }
    } else if (warp >= kWarpGather) {
        // ================================ gather ================================
        // Eight lanes copy the 128 bytes of a row, to the places that the 128-byte swizzle gives
        // them.  Two teams take the stages in turn: a stage's wait, about 200 cycles, comes up every
        // other time (all four warps on every stage: 1.23 ms where this takes 1.12).
        grid_dep_wait();
        const int gt = (int)threadIdx.x - kWarpGather * 32;
        const int team = gt / kGatherTeam, piece = gt & 7, r0 = (gt % kGatherTeam) >> 3;
        RingPos at;
        at.s = team;
        int first = team;
        bool ok = true;
        for (int w = cid; w < n_items && ok; w += nclusters) {
            const Item it = item(w);
            const int hn = it.n >> 1, mine = min(max(it.nt - half * hn, 0), hn);
            uint32_t row[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                row[j] = r0 + 8 * j < mine ? (uint32_t)load_i32(A.row_token + it.row0 + half * hn + r0 + 8 * j) : 0u;
                if (row[j] >= (uint32_t)A.N_x) row[j] = 0;    // (flagged and not stored by the epilogue)
            }
            int k = k_lo + first;
            for (; k < k_hi; k += 2, at.next(A.stages, 2)) {
                if (at.lap > 0 && !pwait(bar(B_EMPTY + at.s), (at.lap - 1) & 1)) {
                    ok = false;
                    break;
                }
                const uint32_t dst = s_base + (uint32_t)(at.s * A.stage_bytes + kABytes + r0 * 128 + ((piece ^ (r0 & 7)) << 4));
                const bool live = k * kKStep + piece * 8 < A.K;
                const uint64_t from = reinterpret_cast<uint64_t>(A.x + piece * 8 + (live ? k * kKStep : 0));
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (r0 + 8 * j < mine)
                        cp_async16(dst + (uint32_t)(j * 8 * 128), from + (uint64_t)row[j] * ((uint32_t)A.K * 2), live);
                cp_async_arrive(bar(B_GATHER + at.s));
            }
            first = k - k_hi;
        }
        cp_async_wait_all();
    } else if (warp == kWarpMma && half != 0) {
        // the odd CTA issues no MMAs
    } else if (warp == kWarpMma) {
        // ================================ even CTA: MMA issuer ================================
        grid_dep_wait();
        const uint64_t da0 = tc::sdesc_sw128(s_base, 16, 1024);
        const uint64_t db0 = tc::sdesc_sw128(s_base + kABytes, 16, 1024);
        const uint16_t pair = (uint16_t)(3u << even);
        // the last lap is not released, so that no arrival reaches a peer that has finished
        long long left = (long long)my_items * (k_hi - k_lo);
        RingPos at;
        bool ok = true, ready = false;
        int i = 0;
        for (int w = cid; w < n_items && ok; w += nclusters) {
            const uint32_t id = tc::idesc(2 * kRowsA, item(w).n, tc::kFmtBF16, 0, 0);
            for (int k0 = k_lo; k0 < k_hi && ok; k0 += part, ++i) {
                const int buf = i & 1, k1 = min(k_hi, k0 + part);
                // both CTAs' epilogues are done with this accumulator
                if (i >= 2 && !pwait(bar(B_ACC_EMPTY + buf), ((i >> 1) - 1) & 1)) {
                    ok = false;
                    break;
                }
                tc::fence_after();
                for (int k = k0; k < k1; ++k) {
                    if (!ready && !pwait(bar(B_FULL + at.s), at.lap & 1)) {
                        ok = false;
                        break;
                    }
                    const RingPos now = at;
                    at.next(A.stages);
                    ready = left > 1 && mbar_test_wait(bar(B_FULL + at.s), at.lap & 1);   // seen while the MMAs are issued
                    tc::fence_after();
                    const uint64_t off = (uint64_t)(now.s * (A.stage_bytes >> 4));
                    tc::mma_pair_bf16_ss_k64_commit(tmem + (uint32_t)(buf * kAccCols), da0 + off, db0 + off, id,
                                                    k > k0 ? 1u : 0u, bar(B_EMPTY + now.s), left > A.stages ? 1u : 0u,
                                                    bar(B_ACC_FULL + buf), k == k1 - 1 ? 1u : 0u, pair);
                    --left;
                    ready = __all_sync(0xffffffffu, ready);
                }
            }
        }
        // every MMA of the pair has completed before TMEM is released
        tc::commit_pair(bar(B_DRAIN));
        __syncwarp();
        (void)mbar_wait_short<200>(bar(B_DRAIN), 0, A.dev_status, nullptr, A.wait_ns);
        __syncwarp();
    } else {
        // ================================ epilogue ================================
        grid_dep_wait();
        const int e8 = (warp - kWarpEpi) >> 2;                // which of every two blocks of 32 tokens
        const int quarter = warp & 3;                         // TMEM lanes this warp may access
        float *stg = reinterpret_cast<float *>(smem + kOffStg + (warp - kWarpEpi) * kStgBytes);
        // the warp that holds the other factor of the same features, and the barrier of the two
        const float *stg_other = reinterpret_cast<const float *>(smem + kOffStg + (e8 * 4 + ((warp - kWarpEpi) & 3 ^ 2)) * kStgBytes);
        const int swap_bar = 1 + e8 * 2 + (quarter & 1);
        const size_t F = (size_t)A.F;
        const int accs = my_items * parts;                    // accumulations in all
        int i = 0;
        bool ok = true;
        // the accumulator of accumulation i is complete / may be written again
        auto acc_full = [&] {
            bool r = mbar_wait_short<200>(bar(B_ACC_FULL + (i & 1)), (uint32_t)((i >> 1) & 1), A.dev_status, abort_flag,
                                           A.wait_ns);
            if (kGated) r = named_all(swap_bar, 64, r);       // the two warps go on together
            ok = __all_sync(0xffffffffu, r);
            tc::fence_after();
            return ok;
        };
        auto release = [&] {
            if (i + 2 >= accs || (A.withhold && i == 0 && half == 1 && warp == kWarpEpi)) return;
            tc::fence_before();
            __syncwarp();
            if (lane == 0) mbar_pair_arrive(bar(B_ACC_EMPTY + (i & 1)), even);   // its MMA warp waits
        };
        // Residual values of the block that comes next, requested as those of the block before it are
        // used: 16 tokens of the lane's feature (h = 0, 1: halves of a block; gated: the half that the
        // warp finishes).  Their rows are on their way into L2 an item ahead.  (8192 x 512 x 4096 fp32
        // with residual 132 us where this takes 54, when each value was requested before its store.)
        constexpr int kHalves = kGated ? 1 : 2;
        uint32_t resid[kResid ? kHalves : 1][kResid ? 16 : 1];
        auto request_residual = [&](const Item &it, int c, int h) {
            const int f0 = (it.fb * 2 + half) * kFeat + (kGated ? quarter & 1 : quarter) * 32;
            const int t0 = c * 32 + (kGated ? (quarter < 2 ? 0 : 16) : 16 * h);
            const inkattn_bf16 *from = A.residual + (size_t)(it.row0 + t0) * F + f0 + lane;
            const int n = f0 + lane < A.F ? it.nt - t0 : 0;
            if (n >= 16) {
#pragma unroll
                for (int j = 0; j < 16; ++j, from += F) resid[h][j] = *from;
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j, from += F)
                    if (j < n) resid[h][j] = *from;
            }
        };
        auto prefetch_residual = [&](const Item &it) {
            const int f0 = (it.fb * 2 + half) * kFeat + (kGated ? quarter & 1 : quarter) * 32;
            if (f0 >= A.F) return;
            for (int t = e8 * 32 + lane; t < it.nt; t += 64) {
                const inkattn_bf16 *from = A.residual + (size_t)(it.row0 + t) * F + f0;
                prefetch_l2(from);
                prefetch_l2(from + min(31, A.F - 1 - f0));
            }
        };
        Item ahead = {};
        bool requested = false;                               // of the next item's first block
        if (kResid && cid < n_items) prefetch_residual(ahead = item(cid));
        for (int w = cid; w < n_items; w += nclusters) {
            const Item it = kResid ? ahead : item(w);
            if (kResid) {
                if (!requested && A.splits == 1 && e8 * 32 < it.nt) {
#pragma unroll
                    for (int h = 0; h < kHalves; ++h) request_residual(it, e8, h);
                }
                requested = false;
                ahead.nt = 0;
                if (w + nclusters < n_items) prefetch_residual(ahead = item(w + nclusters));
            }
            // the warp's 32 features (gated: quarters 0 and 1 hold gates, 2 and 3 the ups of the
            // same features), the lane's feature and its bias
            const int f0 = (it.fb * 2 + half) * kFeat + (kGated ? quarter & 1 : quarter) * 32;
            const int frow = f0 + lane;
            float bias = 0.f;
            if (A.bias && frow < A.F)
                bias = load_f32(A.bias + (size_t)it.e * F * (kGated ? 2 : 1) + (kGated && quarter >= 2 ? F : 0) + frow);
            const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
            const int nblocks = (it.nt + 31) >> 5;
            for (int q = 0; q < parts; ++q, ++i) {
                if (!acc_full()) break;
                if (A.splits > 1 && parts == 1) break;        // (the tile is finished below, from this accumulator)
                if (e8 >= nblocks) release();
                for (int c = e8; c < nblocks; c += 2) {
                    uint32_t v[32];
                    tc::ld32(tmem + (uint32_t)((i & 1) * kAccCols + c * 32) + lanes, v);
                    if (kFine && q > 0) {
                        uint32_t before[32];
                        tc::ld32(t_sums + (uint32_t)(c * 32) + lanes, before);
                        tc::wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            v[j] = __float_as_uint(__uint_as_float(before[j]) + __uint_as_float(v[j]));
                    } else {
                        tc::wait_ld();
                    }
                    if (c + 2 >= nblocks) release();
                    if (kFine && (q < parts - 1 || A.splits > 1)) {
                        tc::st32(t_sums + (uint32_t)(c * 32) + lanes, v);
                        tc::wait_st();
                        continue;
                    }
                    // the block whose residual values are requested as this one's are used
                    const bool more = c + 2 < nblocks;
                    const int c_next = more ? c + 2 : e8;
                    auto request_next = [&](int h) {
                        if (more) request_residual(it, c_next, h);
                        else if (c_next * 32 < ahead.nt) request_residual(ahead, c_next, h);
                    };
                    if (kResid && !more) requested = c_next * 32 < ahead.nt;
                    // tokens of this block that are stored
                    bool mine = c * 32 + lane < it.nt;
                    if (!kResid && A.row_token && mine) {
                        const int t = load_i32(A.row_token + it.row0 + c * 32 + lane);
                        if (t < 0 || t >= A.N_x) {
                            mine = false;
                            set_status(A.dev_status, INKATTN_ERR_DEVICE_BOUNDS);
                        }
                    }
                    const uint32_t live = __ballot_sync(0xffffffffu, mine);
                    // 16 finished tokens t0 .. t0 + 15 of the block, the lane's feature of each, to out
                    // (with one test for all of them where all are stored)
                    auto store16 = [&](const float (&y)[16], int t0) {
                        using Out = std::conditional_t<kFine, float, inkattn_bf16>;
                        const int h = kGated ? 0 : t0 >> 4;
                        Out *to = static_cast<Out *>(A.out) + (size_t)(it.row0 + c * 32 + t0) * F + frow;
                        const uint32_t at = frow < A.F ? live >> t0 & 0xffffu : 0u;
                        auto put = [&](int j) {
                            const float z = kResid ? y[j] + __uint_as_float(resid[h][kResid ? j : 0] << 16) : y[j];
                            if constexpr (kFine) *to = z;
                            else store_bf16(to, z);
                        };
                        if (at == 0xffffu) {
#pragma unroll
                            for (int j = 0; j < 16; ++j, to += F) put(j);
                        } else {
#pragma unroll
                            for (int j = 0; j < 16; ++j, to += F)
                                if ((at >> j) & 1u) put(j);
                        }
                        if (kResid) request_next(h);
                    };
                    float y[16];
                    if (kGated) {
                        // the gate warp finishes the block's first 16 tokens, the up warp the others
                        const int keep = quarter < 2 ? 0 : 16;
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            stg[j * kStgPitch + lane] = __uint_as_float(quarter < 2 ? v[16 + j] : v[j]) + bias;
                        named_sync(swap_bar, 64);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float own = __uint_as_float(quarter < 2 ? v[j] : v[16 + j]) + bias;
                            const float other = stg_other[j * kStgPitch + lane];
                            const float gate = quarter < 2 ? own : other, up = quarter < 2 ? other : own;
                            y[j] = activate<INKATTN_ACT_SILU, kFine>(gate) * up;
                        }
                        named_sync(swap_bar, 64);                 // both have read
                        store16(y, keep);
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) y[j] = activate<kAct, kFine>(__uint_as_float(v[16 * h + j]) + bias);
                            store16(y, 16 * h);
                        }
                    }
                }
            }
            if (!ok || A.splits > 1) break;                   // (of a split: one item)
        }
    }

    if (A.splits > 1) {
        const int et = (int)threadIdx.x - kWarpEpi * 32;
        const bool epi = et >= 0 && et < kEpiThreads && cid < n_items;
        const Item it = only;
        const int share = it.n / A.splits;             // tokens that a pair adds up, a multiple of 8
        __syncwarp();
        cluster_sync();                                // every pair's MMAs are done: the rings are idle
        if (epi) {
            const int quarter = warp & 3;
            const uint32_t place = s_base + (uint32_t)((split * share * kRowsA + quarter * 32 + lane) * 4);
            for (int c = (warp - kWarpEpi) >> 2; c * 32 < it.nt; c += 2) {
                uint32_t v[32];
                tc::ld32((parts > 1 ? t_sums : tmem) + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(c * 32), v);
                tc::wait_ld();
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int t = c * 32 + g * 8, owner = t / share;
                    if (t >= it.nt) break;
                    const uint32_t dst = mapa_shared(place, (uint32_t)(2 * owner + half)) +
                                         (uint32_t)((t - owner * share) * kRowsA * 4);
#pragma unroll
                    for (int j = 0; j < 8; ++j) st_shared_cluster(dst + (uint32_t)(j * kRowsA * 4), v[g * 8 + j]);
                }
            }
        }
        tc::fence_before();
        __syncwarp();
        cluster_sync();                                // every partial tile has arrived, TMEM has been read
        if (warp == kWarpMma) {                        // with the peer CTA's MMA warp
            tc::fence_after();
            tc::tmem_dealloc_pair(tmem, 512);
        }
        if (epi) {
            const size_t F = (size_t)A.F;
            const bool vec = (A.F & 3) == 0;
            // four features of one token per step
            constexpr int kPer = kFeat / 4;            // steps of a token
            const int mine = min(share, it.nt - split * share);
            for (int u = et; u < mine * kPer; u += kEpiThreads) {
                const int t = u / kPer, j = u % kPer;
                const int f = (it.fb * 2 + half) * kFeat + j * 4;
                if (f >= A.F) continue;
                const int i = it.row0 + split * share + t;
                if (A.row_token) {
                    const int s = load_i32(A.row_token + i);
                    if (s < 0 || s >= A.N_x) {
                        if (j == 0) set_status(A.dev_status, INKATTN_ERR_DEVICE_BOUNDS);
                        continue;
                    }
                }
                const float4 *src = reinterpret_cast<const float4 *>(smem) + t * (kRowsA / 4) + j;
                const int step = share * (kRowsA / 4);
                float sum[4] = {}, up[4] = {};
#pragma unroll
                for (int s = 0; s < kMaxSplits; ++s) {
                    if (s >= A.splits) break;
                    const float4 q = src[s * step];
                    sum[0] += q.x; sum[1] += q.y; sum[2] += q.z; sum[3] += q.w;
                    if (kGated) {                      // the ups lie 64 rows on
                        const float4 r = src[s * step + 16];
                        up[0] += r.x; up[1] += r.y; up[2] += r.z; up[3] += r.w;
                    }
                }
                const float *b = A.bias ? A.bias + (size_t)it.e * F * (kGated ? 2 : 1) + f : nullptr;
                const size_t at = (size_t)i * F + f;
                float y[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const bool in = f + n < A.F;
                    y[n] = activate<kGated ? INKATTN_ACT_SILU : kAct, kFine>(sum[n] + (b && in ? load_f32(b + n) : 0.f));
                    if (kGated) y[n] *= up[n] + (b && in ? load_f32(b + F + n) : 0.f);
                }
                if (vec) {
                    if (kResid) {
                        const uint2 r = *reinterpret_cast<const uint2 *>(A.residual + at);
                        y[0] += bf16_lo(r.x); y[1] += bf16_hi(r.x);
                        y[2] += bf16_lo(r.y); y[3] += bf16_hi(r.y);
                    }
                    if (kFine)
                        *reinterpret_cast<float4 *>(static_cast<float *>(A.out) + at) = make_float4(y[0], y[1], y[2], y[3]);
                    else
                        *reinterpret_cast<uint2 *>(static_cast<inkattn_bf16 *>(A.out) + at) =
                            make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
                    continue;
                }
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    if (f + n >= A.F) break;
                    const float o = kResid ? y[n] + load_bf16(A.residual + at + n) : y[n];
                    if (kFine) static_cast<float *>(A.out)[at + n] = o;
                    else store_bf16(static_cast<inkattn_bf16 *>(A.out) + at + n, o);
                }
            }
        }
        return;                                        // (nothing of a peer is read or written after the barrier)
    }

    tc::fence_before();
    __syncthreads();
    if (warp == kWarpMma) {                            // with the peer CTA's MMA warp
        tc::fence_after();
        tc::tmem_dealloc_pair(tmem, 512);
    }
    cluster_sync();                  // a CTA leaves only when no peer writes into it or reads from it
}

namespace {

using Kernel = void (*)(const LinearArgs, const LinearMaps);

template <bool kFine, bool kResid>
Kernel kernel_of(int act) {
    switch (act) {
        case INKATTN_ACT_RELU: return k_linear<INKATTN_ACT_RELU, kFine, kResid>;
        case INKATTN_ACT_GELU: return k_linear<INKATTN_ACT_GELU, kFine, kResid>;
        case INKATTN_ACT_SILU: return k_linear<INKATTN_ACT_SILU, kFine, kResid>;
        case INKATTN_ACT_SWIGLU: return k_linear<INKATTN_ACT_SWIGLU, kFine, kResid>;
        default: return k_linear<INKATTN_ACT_NONE, kFine, kResid>;
    }
}

// Clusters of `ctas` CTAs that are resident at once on the current device `dev` (one CTA per SM;
// every activation's kernel has the same launch shape).
int resident_clusters(int dev, int ctas, int num_sms) {
    static DeviceTable<64, 3> table;
    return table.get(dev, ctas == 2 ? 0 : ctas == 4 ? 1 : 2, [&] {
        int n = 0;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(ctas * (num_sms / ctas > 0 ? num_sms / ctas : 1)), 1, 1);
        cfg.blockDim = dim3(kMaxThreads);
        cfg.dynamicSmemBytes = kSmem;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = (unsigned)ctas;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, k_linear<INKATTN_ACT_NONE, false, false>, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();
            return 0;
        }
        return n;
    });
}

// What a launch would take, in microseconds: the model that picks the token tile and the
// split.  Its constants are fits to measured times of the kernel (GB300, 76 pairs): 19 shapes
// between 1 x 1024 x 1024 and 512 x 8192 x 8192, each with every tile and split.
//   stage   a K = 64 step of a tile of n tokens: the loop of the MMA warp (0.16), the bytes into an
//           SM, which come faster to few of them, or the MMAs
//   finish  an item's epilogue, which overlaps the next item's products
//   join    of a split instead: the partial tiles through distributed shared memory
//   and the weights come from HBM at 7 TB/s at best, 88 GB/s for each SM that asks
double launch_us(long long items, int n, int stages, int splits, int pairs, double weight_bytes) {
    const double busy = fmin((double)(items * splits), (double)pairs);
    const double stage = fmax(fmax(0.16, (16.4 + 0.0655 * n) / (busy <= 40 ? 150.0 : 118.0)), 0.00104 * n);
    const double finish = 0.6 + 0.0071 * n, join = 1.2 + 0.024 * n, start = 1.4 + 0.015 * busy;
    const double item = stages * stage / splits, hbm = weight_bytes / fmin(7.0e6, 0.176e6 * busy);
    if (splits > 1) return start + fmax(item, hbm) + join;
    const double waves = (double)((items + pairs - 1) / pairs);
    return start + fmax(waves * fmax(item, finish), hbm) + fmin(item, finish);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs &args, int act, int num_sms, cudaStream_t stream) {
    if (linear_few(args, act)) return launch_linear_few(args, act, stream);
    LinearArgs a = args;
    const Kernel k = a.residual ? (a.out_f32 ? kernel_of<true, true>(act) : kernel_of<false, true>(act))
                                : (a.out_f32 ? kernel_of<true, false>(act) : kernel_of<false, false>(act));
    cudaError_t err = cudaSuccess;
    for (Kernel f : {k, kernel_of<false, false>(INKATTN_ACT_NONE)})
        if ((err = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem)) != cudaSuccess) return err;
    const int feat = act == INKATTN_ACT_SWIGLU ? 128 : 256, nk = (a.K + kKStep - 1) / kKStep;
    a.n_fblocks = (a.F + feat - 1) / feat;
    a.wait_ns = kernel_debug().wait_ns;
    a.withhold = kernel_debug().withhold;
    // Where the split of the rows among the experts is known on the device alone, the model takes
    // an even one over the experts that can have rows; a tile then leaves room for four times
    // that, so that a busier expert's weights are not read for one small tile after another.
    const long long owners = a.offsets ? (a.E < a.M ? a.E : a.M) : 1;
    const long long rows = (a.M + owners - 1) / owners;
    const double weight_bytes = (double)owners * a.n_fblocks * 2 * kRowsA * a.K * 2;
    int dev = 0;
    if ((err = cudaGetDevice(&dev)) != cudaSuccess) return err;
    auto resident = [&](int ctas) { return resident_clusters(dev, ctas, num_sms); };
    if (resident(2) < 1) return cudaErrorInvalidConfiguration;
    int most_n = a.out_f32 ? kFineN : kMaxN;
    if (a.offsets && 4 * rows < most_n) most_n = rows < 16 ? 64 : (int)(4 * rows + 31) / 32 * 32;
    double best = 0.0;
    long long most_items = 0;
    a.tile_n = 0;
    for (int tile = most_n; tile >= 32; tile -= 32) {
        const long long each = (rows + tile - 1) / tile;                   // tiles of an owner
        const int n = (int)((rows + each - 1) / each + 31) / 32 * 32;
        // items there can be: with experts, full tiles and one more for each that has rows
        const long long bound = (a.offsets ? a.M / tile + owners : each) * a.n_fblocks;
        if (bound > INT_MAX / 2) continue;
        for (int s = 1; s <= kMaxSplits; s *= 2) {
            if (s > 1 && (nk < 2 * s || bound > resident(2 * s))) break;
            const double us = launch_us(owners * each * a.n_fblocks, n, nk, s, resident(2), weight_bytes);
            if (a.tile_n == 0 || us < best) {
                best = us;
                most_items = bound;
                a.tile_n = a.offsets ? tile : n;       // (no larger than the tiles are: the ring gets more stages)
                a.splits = s;
            }
        }
    }
    if (a.tile_n == 0) return cudaErrorInvalidConfiguration;
    a.stage_bytes = kABytes + a.tile_n / 2 * 128;
    a.stages = kRingBytes / a.stage_bytes < kMaxStages ? kRingBytes / a.stage_bytes : kMaxStages;
    const int most = resident(2 * a.splits);
    const int clusters = (int)(most_items < most ? most_items : most);
    LinearMaps maps = {};
    if (!make_linear_maps(a, act == INKATTN_ACT_SWIGLU, &maps)) return cudaErrorInvalidValue;
    if (a.residual && a.row_token) return cudaErrorInvalidValue;   // (no such call)
    const int threads = a.row_token ? kMaxThreads : kThreads;
    return launch_dependent(k, dim3((unsigned)(2 * a.splits * clusters)), dim3((unsigned)threads), kSmem, stream,
                            2 * a.splits, a, maps);
}

}  // namespace inkattn
