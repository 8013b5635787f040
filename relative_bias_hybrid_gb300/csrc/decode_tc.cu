// decode_tc.cu -- split-KV decode on the 5th-generation tensor cores (tcgen05 + TMEM + TMA),
// sm_103a, with the relative-position bias.
//
// [vLLM TML Inkling サポート, §低レイテンシコレクティブとカーネル "FA4 Kernel"] and
// [vLLM hỗ trợ TML Inkling ..., §FA4 với sheared bias]: the attention kernel splits the KV
// length (num_splits picked from batch size, TP size and KV length); the partial results are
// merged afterwards (k_combine in decode.cu).
// [SGLang と Miles が Inkling を初日からサポート, §相対位置バイアス付き Attention]: the logit is
// the scaled dot product plus the bias r_i . P_h[:, i-j] for 0 <= i-j < rel_extent.
//
// One CTA per (split, KV head hk, sequence b).  Its MMA rows are the (token t, query head
// h = hk*g + hh) pairs of the sequence, row = t*g + hh (72 rows for 9 MTP-verify tokens x 8
// heads, padded to 128), so every K/V tile is read once for all the query heads that share
// it.  The Q tile arrives as one 3D TMA box {64 dims, g heads, ql tokens} per half of the
// head dimension, which lands exactly in that row order.  Roles, as in the prefill kernel:
//   warp 0      producer: TMA loads of 128-key K/V tiles (two 64-key cache blocks) of this
//               split's key range into a 4-slot ring, in the order the MMAs consume them
//               (every tile comes from HBM: the ring's depth sets the bytes in flight).
//   warp 1      MMA issuer (the whole warp, one elected lane issuing): S = Q K^T into a
//               double-buffered S in TMEM, O += P V with P (bf16) read from TMEM.
//   warps 2-9   softmax: two warpgroups; row a (TMEM lane a) is shared by one thread of each,
//               which own its key columns [0, 64) and [64, 128).
// TMEM: O [0,128) | S0 [128,256) | S1 [256,384).
//
// Relative bias: only tiles within rel_extent of the queries carry it (the last ones of the
// sequence).  For such a tile the softmax warps first build, per query head, the table
// R[t][x] = r_t . P_h[:, dlo + x] over the tile's 128 + ql distances with mma.sync (one warp
// per head; fp16 operands, fp32 accumulation), then each thread adds its row's 64 entries.
// fp16 keeps 11 significant bits of P (bf16 would keep 8) and represents the bf16 r exactly;
// r is first scaled, per token, by a power of two that keeps it inside fp16's range (exact,
// undone on the fp32 results).  P must lie inside fp16's range (|P| < 65504); a table entry
// that comes out infinite or undefined is flagged as INKATTN_ERR_DEVICE_BOUNDS.  The table holds 16-bit fixed point with one
// step per (head, token) row and round of 72 distances, sigma = (largest |entry| of that
// part of the row) / 32000; the staged bias is within sigma / 2 of the fp32 value.  A tile of the band costs
// four others over a bf16 cache, three over E4M3, 4.5 over 4 bits (L2 round trips for P and 64 table entries a
// thread; 8 sequences x 9 queries, with a bias and without).  Rows of 73 words instead of 72, P in 16-byte
// pieces, loads ahead and one step's factor for most of a half: 64 sequences x 4 queries over 4096 keys, 4
// bits 315 -> 262 us.
// Normalisation: O accumulates P V with P rounded to bf16, and each tile's largest P (its
// row maximum's) is the dominant term whose bf16 rounding matters; that rounding error is
// added to the row's normaliser, while the LSE uses the sum of the fp32 P.
//
// The softmax runs in the log2 domain with the lazy rescale of the prefill kernel (O is
// rescaled only when the running maximum grows by more than 8).  The epilogue writes O / l
// and the natural-log LSE: straight to `out` with one split, else to the split workspace.
#include "common.cuh"
#include "fp8.cuh"
#include "int4.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace inkattn {

namespace {

constexpr int kRows = 128;                 // MMA M: (token, query head) rows, padded
constexpr int kKeys = 128;                 // keys per tile (two cache blocks)
constexpr int kSlotBytes = 32768;          // one MMA operand tile: [d half][128 keys][128 B]
constexpr int kTabW = 144;                 // distances per table row: 128 keys + up to 16 tokens
// Of the 64 keys of a half, at a token t < 16 of table column t + 127 - bb (t + 63 - bb in the second half), those
// that lie on one side of column 72 whatever t.
constexpr int kTabMidLo = 7, kTabMidHi = 54;
constexpr int kTabStride = 146;            // entries from row to row: 73 words, so that a warp's rows spread over the banks
constexpr int kTabRows = kDecodeMaxRows;   // g * ql <= 128

// Three variants, by the cache's element type.  kKv = INKATTN_KV_BF16: TMA loads K/V tiles
// straight into the MMAs' 4-slot ring.  INKATTN_KV_E4M3 and INKATTN_KV_I4: TMA loads tiles of
// codes and their scales into a ring of their own (E4M3 3 slots, 4 bits 6), and converter warps
// (E4M3 six, 4 bits ten) convert Q to f16 in place, then expand each tile (code * scale, exactly)
// to f16 in a 3-slot MMA ring; P is packed as f16, so the MMAs run kind::f16 on f16 operands.
// Warps: 0 TMA, 1 MMA, [2, kWarpSm) converters (codes only), then 8 softmax warps.
//
// What bounds the 4-bit variant: a tile of 128 keys is 17 KB from HBM, a quarter of bf16's, and
// takes about 1950 cycles of an SM, in which the schedulers issue two cycles in three (63%, the busiest
// 65%): 32768 values are expanded, 72 rows of softmax run beside them, and the tensor pipe is active for half.  MTP-verify
// (32 x 9 queries, 32768 keys, band split) 0.54 ms with the combine, bf16 cache 0.66; floor (HBM) 0.17.
// Steps: six warps of 512 threads, 16 units shared out evenly 0.88; ten converter warps with shares by
// their scheduler's load and lane-constant addresses, and rows without a query as zeros instead of masked
// 0.71; the warp index broadcast (uniform registers for the MMA warp, no spills) 0.68; block-table entries
// ahead of the tiles 0.64; a lane for each half's copies 0.60; the warps in two sets that take the tiles in turn
// 0.555; the bias tables' layout and loads below 0.54.  Not kept: pieces taken from a queue in shared memory instead of fixed shares (1.05 for 0.71), the units of a
// tile in a rolled loop (0.69 for 0.60), 4 operand and 3 code slots (no change), the softmax warpgroups each a tile
// of their own in turn, with an O each (0.58 for 0.56), Q as an operand in TMEM (no change), the scales by
// cp.async instead of bulk copies (no change).
template <int kKv>
struct Dec {
    static constexpr bool kCodes = kKv != INKATTN_KV_BF16;
    static constexpr bool kI4 = kKv == INKATTN_KV_I4;
    static constexpr int kThreads = kI4 ? 640 : kCodes ? 512 : 320;
    static constexpr int kWarpSm = kI4 ? 12 : kCodes ? 8 : 2;           // first softmax warp
    static constexpr int kWarpMma = 1;
    // registers a thread at launch, of the warps below kWarpSm, and of the softmax's
    static constexpr int kRegsLaunch = kI4 ? 96 : 128;
    static constexpr int kRegsLow = kI4 ? 64 : 80, kRegsHigh = kI4 ? 144 : 176;
    static_assert(!kCodes || kWarpSm * kRegsLow + 8 * kRegsHigh <= (kWarpSm + 8) * kRegsLaunch,
                  "the split draws on what the block was launched with");
    static constexpr int kConvThreads = kCodes ? (kWarpSm - 2) * 32 : 0;    // converter warps, from 2 on
    static constexpr int kConvArrivals = kI4 ? kConvThreads / 64 : kCodes ? kConvThreads : 1;   // for a tile (4 bits:
                                                             // the warps take turns, and a lane arrives for each)
    static constexpr int kSlots = kCodes ? 3 : 4;            // MMA operand ring
    static constexpr int kCodeSlots = kI4 ? 6 : kCodes ? 3 : 0;      // ring of codes
    static constexpr int kCodeRow = kI4 ? kI4RowBytes : kHeadDim;    // bytes of a row's codes
    static constexpr int kCodeTile = kKeys * kCodeRow;               // one tile: [128 keys][row]
    static constexpr int kCodeSlotBytes = kCodeTile + kKeys * 4;     // + 4 bytes of scales a row
    static constexpr int kOffQ = 0;
    static constexpr int kOffKV = 32768;
    static constexpr int kOffCodes = kOffKV + kSlots * kSlotBytes;
    static constexpr int kOffTab = kOffCodes + kCodeSlots * kCodeSlotBytes;   // 16-bit fixed point [g][ql][kTabStride]
    static constexpr int kOffXchg = kOffTab + kTabRows * kTabStride * 2;     // row maxima / sums
    static constexpr int kOffTsig = kOffXchg + 3 * 2 * kRows * 4;       // fp32 steps [g][ql][2 rounds]
    static constexpr int kOffBar = kOffTsig + kTabRows * 2 * 4;
    // mbarrier indices, laid out from the slot counts
    static constexpr int B_Q = 0;
    static constexpr int B_KV_FULL = 1;
    static constexpr int B_KV_EMPTY = B_KV_FULL + kSlots;
    static constexpr int B_S_FULL = B_KV_EMPTY + kSlots;
    static constexpr int B_P_FULL = B_S_FULL + 2;
    static constexpr int B_PV_DONE = B_P_FULL + 2;
    static constexpr int B_TAB_FULL = B_PV_DONE + 2;
    static constexpr int B_TAB_FREE = B_TAB_FULL + 1;
    static constexpr int B_DRAIN = B_TAB_FREE + 1;
    static constexpr int B_QF = B_DRAIN + 1;                 // codes: Q converted to f16
    static constexpr int B_C_FULL = B_QF + 1;
    static constexpr int B_C_EMPTY = B_C_FULL + kCodeSlots;
    static constexpr int B_COUNT = B_C_EMPTY + kCodeSlots;
    static constexpr int kSmem = kOffBar + B_COUNT * 8 + 16;
    static_assert(kSmem <= 232448, "shared memory budget");
    static_assert(kOffKV % 1024 == 0 && kOffCodes % 1024 == 0 && kCodeSlotBytes % (kI4 ? 512 : 128) == 0,
                  "alignment of the rings (the 64-byte swizzle of 4-bit tiles repeats every 512 bytes)");
    static_assert(kOffTab % 16 == 0 && kOffBar % 8 == 0, "alignment of the table and the barriers");
    static_assert(kThreads == 32 * (kWarpSm + 8), "eight softmax warps last");
};

// The 4-bit variant's shares: the units of a tile (16) that each warp expands, a hexadecimal digit for warp 0 on,
// by how many lane quarters have rows; more of them where the warp's scheduler (warp % 4) has
// softmax warps without rows to work on.  Five warps take the tiles 0, 2, ... of the ring, the other five
// 1, 3, ...: a warp then waits and arrives half as often for the same units (MTP-verify 0.56 ms; all ten for
// every tile 0.60, of that with equal shares 0.64).
constexpr int kUnitsMax = 6;               // of a warp
constexpr uint64_t kEven1 = 0x4040014300ull, kOdd1 = 0x440203300000ull, kEven2 = 0x2040024400ull, kOdd2 = 0x530204200000ull,
                   kEven3 = 0x3050024200ull, kOdd3 = 0x620203300000ull, kEven4 = 0x3030043300ull, kOdd4 = 0x430302400000ull;
// Whether each unit of a tile is expanded once, the even tiles' by the warps of ~odd and the odd ones' by those of odd.
constexpr bool share_holds(uint64_t even_share, uint64_t odd_share, uint32_t odd) {
    const uint64_t share[2] = {even_share, odd_share};
    int units[2] = {0, 0}, warps[2] = {0, 0};
    for (int w = 0; w < 16; ++w)
        for (int i = 0; i < 2; ++i) {
            const int u = (int)(share[i] >> (4 * w)) & 15;
            if (u > kUnitsMax) return false;
            if (u > 0 && (w < 2 || w >= Dec<INKATTN_KV_I4>::kWarpSm || (int)(odd >> w & 1) != i)) return false;
            units[i] += u;
            warps[i] += u > 0;
        }
    return units[0] == 16 && units[1] == 16 && warps[0] == Dec<INKATTN_KV_I4>::kConvArrivals && warps[1] == warps[0];
}
constexpr uint32_t kOddWarps = 1u << 5 | 1u << 6 | 1u << 8 | 1u << 10 | 1u << 11;
static_assert(share_holds(kEven1, kOdd1, kOddWarps) && share_holds(kEven2, kOdd2, kOddWarps) &&
              share_holds(kEven3, kOdd3, kOddWarps) && share_holds(kEven4, kOdd4, kOddWarps), "each unit of a tile once, by the warps that arrive for it");

constexpr uint32_t kTmemO = 0, kTmemS0 = 128;
constexpr int kBarPair = 8;                // named barriers 8-11: the softmax row pairs, per lane quarter

struct DecTcArgs {
    inkattn_attn_params p;
    float scale;            // softmax scale
    int S;                  // number of splits
    int band_split;         // S == 2 cut at the band's start; the grid is (Hkv, B, 2)
    int ql;                 // rows of the Q box per head (max_seqlen_q)
    float *ws_o;
    float *ws_lse;
    long long kv_rows;      // rows of the cache tensor maps (OOB row = this)
    uint64_t wait_ns;       // limit of every bounded wait
    int withhold;           // failure-path test: the softmax withholds its first P arrival
    uint32_t i4_mask, i4_exponent;   // i4_decode8's constants
};

}  // namespace

template <int kKv>
__global__ void __launch_bounds__(Dec<kKv>::kThreads, 1)
k_decode_tc(const DecTcArgs A, const __grid_constant__ CUtensorMap qmap,
            const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ __align__(1024) unsigned char smem[];
    grid_dep_wait();                                   // q and the cache: written by the prologue
    using C = Dec<kKv>;
    constexpr bool kCodes = C::kCodes;
    const inkattn_attn_params &p = A.p;
    // band split: the CTAs of split 0 (the keys before the band) come first in the grid, so
    // that the short split-1 CTAs run on the SMs the streaming ones leave free
    const int split = A.band_split ? (int)blockIdx.z : (int)blockIdx.x;
    const int hk = A.band_split ? (int)blockIdx.x : (int)blockIdx.y;
    const int b = A.band_split ? (int)blockIdx.y : (int)blockIdx.z;
    // (broadcast, so that the compiler knows the roles' branches to be uniform over a warp and keeps the MMA
    // warp's descriptors in uniform registers: without it an MMA of the variants with codes takes
    // 100 cycles to issue instead of 40)
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int g = p.Hq / p.Hkv;

    // ---- sequence geometry and this split's key range (uniform over the CTA)
    const int start = p.cu_seqlens_q[b], end = p.cu_seqlens_q[b + 1];
    const int T = p.seqlen_k[b];
    const int q_len = end - start;
    if (start < 0 || end < start || end > p.N_tok || q_len > A.ql || T < q_len ||
        T > p.max_seqlen_k || q_len * g > kRows) {
        if (threadIdx.x == 0) set_status(p.dev_status, INKATTN_ERR_DEVICE_BOUNDS);
        return;
    }
    if (q_len == 0) return;
    const int n_rows = q_len * g;
    const int pos0 = T - q_len;                       // position of token 0
    int blk_first = 0;
    if (p.window > 0) blk_first = max(0, pos0 - p.window + 1) / kBlock;
    const int blk_end = (T + kBlock - 1) / kBlock;    // exclusive
    const int nblk = blk_end - blk_first;
    int my_lo, my_hi;
    if (A.band_split) {
        // two parts: the keys before the band, in whole 128-key tiles, and the rest (the keys
        // within rel_extent of the first query, whose tiles build bias tables)
        const int band_key_lo = max(0, pos0 - p.rel_extent + 1);
        const int cut = blk_first + ((max(blk_first, min(blk_end, band_key_lo / kBlock)) - blk_first) & ~1);
        my_lo = split == 0 ? blk_first : cut;
        my_hi = split == 0 ? cut : blk_end;
    } else if (C::kI4) {
        // parts of equal cost in whole tiles, a block of the band counting kI4BandCost others: with few
        // sequences the CTAs of the band would be the last by far
        const int band = p.rel_extent > 0 ? max(blk_first, min(blk_end, max(0, pos0 - p.rel_extent + 1) / kBlock)) : blk_end;
        const int before = band - blk_first;
        const long long cost = before + (long long)kI4BandCost * (blk_end - band);
        auto cut = [&](int part) {
            const int at = (int)(part * cost / A.S);
            return blk_first + min(nblk, ((at <= before ? at : before + (at - before) / kI4BandCost) + 1) & ~1);
        };
        my_lo = cut(split);
        my_hi = split == A.S - 1 ? blk_end : cut(split + 1);
    } else {
        const int per = (nblk + A.S - 1) / A.S;
        my_lo = blk_first + split * per;
        my_hi = min(blk_end, my_lo + per);
    }
    const int my_n = max(0, my_hi - my_lo);
    const int N = (my_n + 1) / 2;                     // 128-key tiles
    const int kr_lo = my_lo * kBlock, kr_hi = my_hi * kBlock;
    const int g_shift = (g & (g - 1)) == 0 ? __ffs(g) - 1 : -1;

    if (N == 0) {
        // an empty split: its partial result is empty (O = 0, LSE = -inf)
        for (int idx = threadIdx.x; idx < n_rows * (kHeadDim / 4); idx += C::kThreads) {
            const int row = idx / (kHeadDim / 4), c4 = idx - row * (kHeadDim / 4);
            const int t = g_shift >= 0 ? row >> g_shift : row / g, hh = row - t * g;
            const size_t qrow = (size_t)(start + t) * p.Hq + hk * g + hh;
            *reinterpret_cast<float4 *>(A.ws_o + (qrow * A.S + split) * kHeadDim + c4 * 4) =
                make_float4(0.f, 0.f, 0.f, 0.f);
            if (c4 == 0) A.ws_lse[qrow * A.S + split] = -INFINITY;
        }
        return;
    }

    const uint32_t s_base = smem_u32(smem);
    if ((s_base & 1023u) != 0u) {
        if (threadIdx.x == 0) set_status(p.dev_status, INKATTN_ERR_DEVICE_BOUNDS);
        return;
    }
    auto bar = [&](int i) { return s_base + C::kOffBar + 8u * (uint32_t)i; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffBar + C::B_COUNT * 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffBar + C::B_COUNT * 8 + 4);
    auto wwait = [&](uint32_t addr, uint32_t parity) -> bool {
        const bool r = mbar_wait(addr, parity, p.dev_status, abort_flag, A.wait_ns);
        return __all_sync(0xffffffffu, r);
    };

    if (threadIdx.x == 0) {
        mbar_init(bar(C::B_Q), 1);
        for (int s = 0; s < C::kSlots; ++s) {
            mbar_init(bar(C::B_KV_FULL + s), C::kConvArrivals);        // tile converters, or the TMA
            mbar_init(bar(C::B_KV_EMPTY + s), 1);
        }
        if constexpr (kCodes) {
            mbar_init(bar(C::B_QF), C::kConvThreads);
            for (int s = 0; s < C::kCodeSlots; ++s) {
                mbar_init(bar(C::B_C_FULL + s), 1);
                mbar_init(bar(C::B_C_EMPTY + s), C::kConvArrivals);
            }
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(C::B_S_FULL + s), 1);
            mbar_init(bar(C::B_P_FULL + s), 256);
            mbar_init(bar(C::B_PV_DONE + s), 1);
        }
        mbar_init(bar(C::B_TAB_FULL), 256);
        mbar_init(bar(C::B_TAB_FREE), 256);
        mbar_init(bar(C::B_DRAIN), 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == C::kWarpMma) {
        tc::tmem_alloc(smem_u32(tmem_slot), 512);
        tc::tmem_relinquish();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;

    const float lam = (p.log_scale_base > 1.f) ? fmaxf(1.f, logf((float)T) / logf(p.log_scale_base)) : 1.f;
    const float c_qk = lam * A.scale * kLog2e;       // S (with the bias folded in) -> log2 logit
    const float inv_scale = 1.f / A.scale;           // bias in S units

    // Variants with codes: the warpgroups of the TMA, MMA and converter warps give registers to the
    // two softmax warpgroups.
    if (warp == 0) {
        // ================================ producer ================================
        if constexpr (kCodes) tc::reg_dealloc<C::kRegsLow>();
        bool ok = true;
        if (lane == 0) {
            tma_prefetch_desc(&qmap);
            tma_prefetch_desc(&kmap);
            tma_prefetch_desc(&vmap);
            const uint32_t qbytes = (uint32_t)(2 * 64 * 2 * g * A.ql);
            mbar_arrive_expect_tx(bar(C::B_Q), qbytes);
            tma_load_3d(s_base + C::kOffQ, &qmap, 0, hk * g, start, bar(C::B_Q));
            tma_load_3d(s_base + C::kOffQ + 16384, &qmap, 64, hk * g, start, bar(C::B_Q));
        }
        // the ring the TMA fills: the MMAs' own (bf16 cache) or that of codes
        constexpr int kRing = kCodes ? C::kCodeSlots : C::kSlots;
        constexpr int kRingFull = kCodes ? C::B_C_FULL : C::B_KV_FULL;
        constexpr int kRingEmpty = kCodes ? C::B_C_EMPTY : C::B_KV_EMPTY;
        int kv_loads = 0;
        // Block-table entries, 32 at a time, one a lane, and the next 32 already asked for: the tiles of
        // a 4-bit cache come faster than a round trip to memory for each.  -2: past this split's range.
        auto entries = [&](int first) -> int {
            const int lb = first + lane;                     // logical cache block
            return lb >= my_hi ? -2
                 : lb < p.max_blocks_per_seq ? load_i32(p.block_table + (size_t)b * p.max_blocks_per_seq + lb) : -1;
        };
        int tab_first = my_lo, tab = entries(my_lo), tab_next = entries(my_lo + 32);
        auto tile_blocks = [&](int n) -> int2 {              // of tile n, in ascending order
            const int at = my_lo + 2 * n;
            if (at >= tab_first + 32) {
                tab_first += 32;
                tab = tab_next;
                tab_next = entries(tab_first + 32);
            }
            return make_int2(__shfl_sync(0xffffffffu, tab, at - tab_first),
                             __shfl_sync(0xffffffffu, tab, at - tab_first + 1));
        };
        auto load_kv = [&](int2 blocks, int isv) -> bool {
            const int L = kv_loads++, slot = L % kRing;
            const int blk[2] = {blocks.x, blocks.y};
            if (L >= kRing && !wwait(bar(kRingEmpty + slot), ((L / kRing) - 1) & 1)) {
                --kv_loads;                                  // not issued
                return false;
            }
            const void *map = isv ? static_cast<const void *>(&vmap) : static_cast<const void *>(&kmap);
            long long row[2];
            bool have[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                row[half] = A.kv_rows;                       // past the tensor: TMA fills zeros
                have[half] = blk[half] >= 0 && blk[half] < p.num_blocks;
                if (have[half]) row[half] = ((long long)blk[half] * p.Hkv + hk) * kBlock;
            }
            if constexpr (!kCodes) {
                if (lane == 0) {
                    const uint32_t dst = s_base + C::kOffKV + slot * kSlotBytes;
                    const uint32_t fb = bar(C::B_KV_FULL + slot);
                    mbar_arrive_expect_tx(fb, kSlotBytes);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        if (blk[half] != -2 && !have[half]) set_status(p.dev_status, INKATTN_ERR_DEVICE_BOUNDS);
                        tma_load_2d(dst + half * 8192, map, 0, (int)row[half], fb);
                        tma_load_2d(dst + 16384 + half * 8192, map, 64, (int)row[half], fb);
                    }
                }
            } else {
                // codes of 128 keys, then 4 bytes of scales for each; a half without a loaded
                // block reads as zero codes (TMA fill) with zero scales (written here)
                unsigned char *slot_p = smem + C::kOffCodes + slot * C::kCodeSlotBytes;
                uint32_t *sc = reinterpret_cast<uint32_t *>(slot_p + C::kCodeTile);
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    if (!have[half]) {
                        sc[half * 64 + lane] = 0u;
                        sc[half * 64 + 32 + lane] = 0u;
                    }
                __syncwarp();
                const uint32_t fb = bar(C::B_C_FULL + slot);
                if (lane == 0) mbar_arrive_expect_tx(fb, C::kCodeTile + 256u * (uint32_t)(have[0] + have[1]));
                __syncwarp();
                if (lane < 2) {                              // a lane for each half: its copies go out beside the other's
                    const int half = lane;
                    const bool mine = half == 0 ? have[0] : have[1];
                    const long long at = half == 0 ? row[0] : row[1];
                    const uint32_t dst = smem_u32(slot_p);
                    const float *scales = isv ? p.v_scale : p.k_scale;
                    if ((half == 0 ? blk[0] : blk[1]) != -2 && !mine) set_status(p.dev_status, INKATTN_ERR_DEVICE_BOUNDS);
                    tma_load_2d(dst + half * (C::kCodeTile / 2), map, 0, (int)at, fb);
                    if (mine) bulk_load(dst + C::kCodeTile + half * 256, scales + at, 256u, fb);
                }
            }
            __syncwarp();
            return true;
        };
        // consumption order of the MMA warp: K_0, then per tile n >= 1: K_n, V_{n-1}; then V_{N-1}
        int2 behind = tile_blocks(0);
        ok = load_kv(behind, 0);
        for (int n = 1; n < N && ok; ++n) {
            const int2 blocks = tile_blocks(n);
            ok = load_kv(blocks, 0);
            if (ok) ok = load_kv(behind, 1);
            behind = blocks;
        }
        if (ok) ok = load_kv(behind, 1);
        // nothing may still be landing in shared memory when the CTA tears down, also when a
        // role gave up: the copies issued and not yet consumed are the last kRing
        if (lane == 0) {
            mbar_drain(bar(C::B_Q), 0, p.dev_status, A.wait_ns);
            for (int L = max(0, kv_loads - kRing); L < kv_loads; ++L)
                mbar_drain(bar(kRingFull + L % kRing), (L / kRing) & 1, p.dev_status, A.wait_ns);
        }
    } else if (warp == C::kWarpMma) {
        // ================================ MMA issuer ================================
        if constexpr (kCodes) tc::reg_dealloc<C::kRegsLow>();
        constexpr uint32_t kFmt = kCodes ? tc::kFmtF16 : tc::kFmtBF16;   // both operands alike
        const uint32_t id_qk = tc::idesc(128, 128, kFmt, 0, 0);
        const uint32_t id_pv = tc::idesc(128, 128, kFmt, 0, 1);
        // the whole warp runs this loop with the same values in every lane (the MMAs and
        // commits are warp-collective); per-slot descriptors differ only in the start address
        // field, which stays below its 14 bits (shared memory < 256 KB)
        const uint64_t dq = tc::sdesc_sw128(s_base + C::kOffQ, 16, 1024);
        const uint64_t dk0 = tc::sdesc_sw128(s_base + C::kOffKV, 16, 1024);
        const uint64_t dv0 = tc::sdesc_sw128(s_base + C::kOffKV, 16384, 1024);
        auto slot_off = [](int slot) { return (uint64_t)(slot * (kSlotBytes >> 4)); };
        bool ok = wwait(bar(kCodes ? C::B_QF : C::B_Q), 0);   // (codes: Q once converted to f16)
        int kv_used = 0;
        auto next_tile = [&](int &slot, bool &last) -> bool {
            const int L = kv_used++;
            slot = L % C::kSlots;
            last = L + C::kSlots >= 2 * N;
            return wwait(bar(C::B_KV_FULL + slot), (L / C::kSlots) & 1);
        };
        auto issue_pv = [&](int m) -> bool {
            if (!wwait(bar(C::B_P_FULL + (m & 1)), (m >> 1) & 1)) return false;
            int slot;
            bool last;
            if (!next_tile(slot, last)) return false;
            // keys at or past the sequence end inside a loaded block: zero their V rows so
            // that P = 0 there contributes exact zeros whatever the cache slots hold
            const int j0 = kr_lo + m * kKeys;
            const int nvalid = max(0, min(kKeys, T - j0));
            const int nload = min(kKeys, (my_hi - my_lo - 2 * m) * kBlock);
            if (nvalid < nload) {
                unsigned char *vp = smem + C::kOffKV + slot * kSlotBytes;
                const int rows = nload - nvalid;
                for (int idx = lane; idx < rows * 16; idx += 32) {
                    const int key = nvalid + idx / 16, dh = (idx >> 3) & 1, ch = idx & 7;
                    *reinterpret_cast<uint4 *>(vp + dh * 16384 + (key >> 6) * 8192 + (key & 63) * 128 + ch * 16) =
                        make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
            tc::fence_after();
            tc::mma_bf16_ts_k128_commit<false>(tmem + kTmemO, tmem + kTmemS0 + (uint32_t)(m & 1) * 128,
                                               dv0 + slot_off(slot), id_pv, m > 0 ? 1u : 0u, bar(C::B_PV_DONE + (m & 1)),
                                               bar(C::B_KV_EMPTY + slot), last ? 0u : 1u);
            __syncwarp();
            return true;
        };
        for (int n = 0; n < N && ok; ++n) {
            int slot;
            bool last;
            ok = next_tile(slot, last);
            if (!ok) break;
            tc::fence_after();
            tc::mma_bf16_ss_k128_commit<false>(tmem + kTmemS0 + (uint32_t)(n & 1) * 128, dq, dk0 + slot_off(slot),
                                               id_qk, 0u, bar(C::B_S_FULL + (n & 1)), bar(C::B_KV_EMPTY + slot),
                                               last ? 0u : 1u);
            __syncwarp();
            if (n >= 1) ok = issue_pv(n - 1);
        }
        if (ok) ok = issue_pv(N - 1);
        // every MMA of this CTA has completed before TMEM is released (also after a role gave up)
        tc::commit(bar(C::B_DRAIN));
        __syncwarp();
        (void)mbar_drain(bar(C::B_DRAIN), 0, p.dev_status, A.wait_ns);
        __syncwarp();
    } else if (kCodes && warp < C::kWarpSm) {
        // ================================ converters (caches of codes) ================================
        if constexpr (kCodes) tc::reg_dealloc<C::kRegsLow>();
        // Q first, then the K/V tiles
        const int ct = threadIdx.x - 32 - (warp > C::kWarpMma ? 32 : 0);   // 0 .. kConvThreads - 1
        bool ok = wwait(bar(C::B_Q), 0);
        if (ok) {
            uint4 *qw = reinterpret_cast<uint4 *>(smem + C::kOffQ);
            uint32_t most = 0;                                // the largest |q|, as bf16 bits, in each half
            for (int i = ct; i < 32768 / 16; i += C::kConvThreads) {
                // rows without a query are zeros, and so are their logits: they then need no mask
                // (16-byte pieces of a row, 8 in each half of the head dimension)
                const uint4 w = ((i >> 3) & (kRows - 1)) < n_rows ? qw[i] : make_uint4(0, 0, 0, 0);
                qw[i] = make_uint4(pack_f16(bf16_lo(w.x), bf16_hi(w.x)), pack_f16(bf16_lo(w.y), bf16_hi(w.y)),
                                   pack_f16(bf16_lo(w.z), bf16_hi(w.z)), pack_f16(bf16_lo(w.w), bf16_hi(w.w)));
                most = max_u16x2(max_u16x2(most, max_u16x2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu)),
                                 max_u16x2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
            }
            fence_proxy_async_smem();
            mbar_arrive(bar(C::B_QF));
            // 65280 is the last bf16 number inside fp16's range
            if (max(most & 0xFFFFu, most >> 16) > 0x477Fu) set_status(p.dev_status, INKATTN_ERR_DEVICE_BOUNDS);
        }
        auto tile_of = [&](int L) { return L == 0 ? 0 : L == 2 * N - 1 ? N - 1 : (L & 1) ? (L + 1) >> 1 : (L >> 1) - 1; };
        if constexpr (C::kI4) {
            // A tile is 16 units of 16 keys x two groups of 32 values (a half of the head dimension): a
            // lane takes one key's group, its 16 bytes (the TMA's 64-byte swizzle spreads eight keys
            // over the banks) to four chunks of 16 bytes (the MMA's 128-byte swizzle does the same).
            // Both swizzles depend on the lane alone, so a unit's addresses are the lane's plus the
            // unit's.
            // A warp has the same units of every other tile.
            const int odd = (int)(kOddWarps >> warp) & 1;
            const uint64_t share = odd ? (n_rows <= 32 ? kOdd1 : n_rows <= 64 ? kOdd2 : n_rows <= 96 ? kOdd3 : kOdd4)
                                       : (n_rows <= 32 ? kEven1 : n_rows <= 64 ? kEven2 : n_rows <= 96 ? kEven3 : kEven4);
            int u0 = 0;
            for (int i = 0; i < warp; ++i) u0 += (int)(share >> (4 * i)) & 15;
            const int units = (int)(share >> (4 * warp)) & 15;
            const int k16 = lane & 15, grp = lane >> 4;
            const uint32_t src_lane = (uint32_t)(k16 * kI4RowBytes + ((grp ^ ((k16 >> 1) & 3)) << 4));
            const uint32_t byte_lane = (uint32_t)(C::kCodeTile + k16 * kI4RowScales + grp);
            uint32_t dst_lane[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) dst_lane[c] = (uint32_t)(k16 * 128 + (((grp * 4 + c) ^ (k16 & 7)) << 4));
            constexpr int kTogether = 3;
            int s4 = odd, s16 = odd;
            uint32_t turn4 = 0, turn16 = 0;                   // of the rings: parity of the waits
            bool bad = false;
            for (int L = odd; L < 2 * N; L += 2) {
                if (!(ok = wwait(bar(C::B_C_FULL + s4), turn4))) break;
                if (L >= C::kSlots && !(ok = wwait(bar(C::B_KV_EMPTY + s16), turn16 ^ 1u))) break;
                const uint32_t src = s_base + C::kOffCodes + s4 * C::kCodeSlotBytes;
                const uint32_t dst = s_base + C::kOffKV + s16 * kSlotBytes;
                const int key_end = min(T, kr_hi) - (kr_lo + tile_of(L) * kKeys);
#pragma unroll
                for (int first = 0; first < kUnitsMax; first += kTogether) {
                    if (first >= units) break;
                    uint4 w[kTogether];
                    uint32_t byte[kTogether];
#pragma unroll
                    for (int i = 0; i < kTogether; ++i) {     // (their loads go out together)
                        if (first + i >= units) break;
                        const int kb = (u0 + first + i) & 7, half = (u0 + first + i) >> 3;
                        w[i] = lds_u32x4(src + kb * (16 * kI4RowBytes) + (src_lane ^ (half << 5)));
                        byte[i] = lds_u8(src + kb * (16 * kI4RowScales) + 2 * half + byte_lane);
                        if (kb * 16 + k16 >= key_end) byte[i] = 0;
                    }
#pragma unroll
                    for (int i = 0; i < kTogether; ++i) {
                        if (first + i >= units) break;
                        const int kb = (u0 + first + i) & 7, half = (u0 + first + i) >> 3;
                        const bool over = byte[i] > kI4ScaleMax;
                        bad |= over;
                        const I4Scale f = i4_factors(over ? 0u : byte[i]);
                        const uint32_t to = dst + half * 16384 + kb * 2048;
                        sts_u32x4(to + dst_lane[0], i4_decode8(w[i].x, f, A.i4_mask, A.i4_exponent));
                        sts_u32x4(to + dst_lane[1], i4_decode8(w[i].y, f, A.i4_mask, A.i4_exponent));
                        sts_u32x4(to + dst_lane[2], i4_decode8(w[i].z, f, A.i4_mask, A.i4_exponent));
                        sts_u32x4(to + dst_lane[3], i4_decode8(w[i].w, f, A.i4_mask, A.i4_exponent));
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(C::B_C_EMPTY + s4));
                    mbar_arrive(bar(C::B_KV_FULL + s16));
                }
                if ((s4 += 2) >= C::kCodeSlots) s4 -= C::kCodeSlots, turn4 ^= 1u;
                if ((s16 += 2) >= C::kSlots) s16 -= C::kSlots, turn16 ^= 1u;
            }
            if (bad) set_status(p.dev_status, INKATTN_ERR_DEVICE_BOUNDS);
        }
        for (int L = 0; !C::kI4 && L < 2 * N && ok; ++L) {
            const int n = tile_of(L);
            constexpr int kRing = kCodes ? C::kCodeSlots : 1;    // (the bf16 variant has no such warps)
            const int s8 = L % kRing, s16 = L % C::kSlots;
            if (!(ok = wwait(bar(C::B_C_FULL + s8), (L / kRing) & 1))) break;
            if (L >= C::kSlots && !(ok = wwait(bar(C::B_KV_EMPTY + s16), ((L / C::kSlots) - 1) & 1))) break;
            const unsigned char *src = smem + C::kOffCodes + s8 * C::kCodeSlotBytes;
            unsigned char *dst = smem + C::kOffKV + s16 * kSlotBytes;
            const int key_end = min(T, kr_hi) - (kr_lo + n * kKeys);
            bool bad = false;
            const float *sc = reinterpret_cast<const float *>(src + C::kCodeTile);
            for (int it = ct; it < kKeys * 8; it += 192) {
                const int key = it >> 3, j16 = it & 7, sw = key & 7;
                const uint4 w = *reinterpret_cast<const uint4 *>(src + key * 128 + j16 * 16);
                float sv = key < key_end ? sc[key] : 0.f;
                const bool good = sv == 0.f || (sv >= 0x1p-24f && sv <= 128.f);
                bad |= !good;
                const __half2 s2 = __float2half2_rn(good ? sv : 0.f);
                const int base = (j16 >> 2) * 16384 + key * 128;
                *reinterpret_cast<uint4 *>(dst + base + ((((j16 & 3) * 2) ^ sw) << 4)) =
                    make_uint4(e4m3x2_to_f16x2_scaled(w.x, s2), e4m3x2_to_f16x2_scaled(w.x >> 16, s2),
                               e4m3x2_to_f16x2_scaled(w.y, s2), e4m3x2_to_f16x2_scaled(w.y >> 16, s2));
                *reinterpret_cast<uint4 *>(dst + base + ((((j16 & 3) * 2 + 1) ^ sw) << 4)) =
                    make_uint4(e4m3x2_to_f16x2_scaled(w.z, s2), e4m3x2_to_f16x2_scaled(w.z >> 16, s2),
                               e4m3x2_to_f16x2_scaled(w.w, s2), e4m3x2_to_f16x2_scaled(w.w >> 16, s2));
            }
            if (bad) set_status(p.dev_status, INKATTN_ERR_DEVICE_BOUNDS);
            fence_proxy_async_smem();
            mbar_arrive(bar(C::B_C_EMPTY + s8));
            mbar_arrive(bar(C::B_KV_FULL + s16));
        }
    } else {
        // ================================ softmax ================================
        if constexpr (kCodes) tc::reg_alloc<C::kRegsHigh>();
        const int quad = warp & 3;
        const int sw = warp - C::kWarpSm;                     // softmax warp index 0..7
        const int hw = sw >> 2;                               // column half
        const int a = quad * 32 + lane;                       // MMA row = TMEM lane
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
        const bool valid_row = a < n_rows;
        const bool quad_live = quad * 32 < n_rows;            // uniform over the warp (and its pair)
        const int t = valid_row ? (g_shift >= 0 ? a >> g_shift : a / g) : 0;
        const int hh = a - t * g;
        const int i_pos = pos0 + t;
        const int cb = 64 * hw;
        unsigned short *tab = reinterpret_cast<unsigned short *>(smem + C::kOffTab);
        float *tsig = reinterpret_cast<float *>(smem + C::kOffTsig);
        float *xchg = reinterpret_cast<float *>(smem + C::kOffXchg);
        // The two threads of a row meet on a named barrier of the row's lane quarter (64
        // threads, one warp of each column half), as in the prefill kernel: every thread
        // makes exactly N + 1 meetings (warps whose rows are all padding skip their tiles'
        // meetings and make them up at the end, as a thread that left the loop early does).
        auto pair_meet = [&]() { asm volatile("bar.sync %0, 64;" :: "r"(kBarPair + quad) : "memory"); };
        int met = 0;
        const bool has_bias = p.rel_extent > 0;
        const int gq = lane >> 2, tq = lane & 3;              // mma.sync fragment coordinates
        int band_round = 0;
        bool ok = true;

        float m_run = -INFINITY, l_run = 0.f;   // l_run: sum of the fp32 P (for the LSE)
        float lc_run = 0.f;                      // bf16 rounding of each tile's largest P (normaliser)
        auto wait_pv = [&](int m) -> bool { return wwait(bar(C::B_PV_DONE + (m & 1)), (m >> 1) & 1); };
        for (int n = 0; n < N; ++n) {
            const int j0 = kr_lo + n * kKeys;
            const bool band = has_bias && (pos0 - (j0 + kKeys - 1) < p.rel_extent);
            const int dlo = pos0 - j0 - (kKeys - 1);          // distance at table column 0
            if (band) {
                // ---- relative rows of this tile, one query head per warp, into the table
                if (band_round > 0 && !(ok = wwait(bar(C::B_TAB_FREE), (band_round - 1) & 1))) break;
                for (int hq = sw; hq < g; hq += 8) {
                    const int h = hk * g + hq;
                    const float *Ph = p.P + (size_t)h * p.rel_extent * 32;
                    const inkattn_bf16 *rh = p.r + ((size_t)start * p.Hq + h) * 32;
                    // d_r = 32 (checked on the host): two k steps of 16.  A fragments: tokens gq
                    // (e even) and gq + 8 (e odd), each lane 8 of a token's 32 features; the four
                    // lanes of a token (tq = 0..3) hold all of them.
                    // (Which column a k stands for is free as long as r and P agree: a lane has the columns
                    // 16 kk + 4 tq .. + 3 of a step, 16 bytes of P, so that a row's 128 bytes take two accesses.)
                    // The first round's P is asked for before r is waited for, the second's before the first is
                    // stored (bf16, whose softmax has the registers) or right behind.
                    constexpr int kGrp = 9;
                    static_assert(kTabW / 8 == 2 * kGrp, "two rounds");
                    float4 raw[kGrp][2];
                    auto ask = [&](int rd) {
#pragma unroll
                        for (int u = 0; u < kGrp; ++u) {
                            const int dl = dlo + (rd * kGrp + u) * 8 + gq;
                            const bool dv = dl >= 0 && dl < p.rel_extent;
#pragma unroll
                            for (int kk = 0; kk < 2; ++kk)
                                raw[u][kk] = dv ? __ldg(reinterpret_cast<const float4 *>(Ph + (size_t)dl * 32 + kk * 16 + 4 * tq))
                                                : make_float4(0.f, 0.f, 0.f, 0.f);
                        }
                    };
                    ask(0);
                    float rv[2][4][2];
                    float rm[2] = {0.f, 0.f};
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int tt = gq + ((e & 1) << 3);
                            const int col = kk * 16 + 4 * tq + (e >> 1) * 2;
                            const uint32_t w2 = tt < q_len
                                ? load_u32(rh + (size_t)tt * 32 * p.Hq + col)
                                : 0u;
                            rv[kk][e][0] = bf16_lo(w2);
                            rv[kk][e][1] = bf16_hi(w2);
                            rm[e & 1] = fmaxf(rm[e & 1], fmaxf(fabsf(rv[kk][e][0]), fabsf(rv[kk][e][1])));
                        }
                    float rsc[2], rusc[2];                     // per token row: fp16 prescale and its inverse
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        rm[i] = fmaxf(rm[i], __shfl_xor_sync(0xffffffffu, rm[i], 1));
                        rm[i] = fmaxf(rm[i], __shfl_xor_sync(0xffffffffu, rm[i], 2));
                        rsc[i] = fp16_prescale(rm[i]);
                        rusc[i] = 1.f / rsc[i];
                    }
                    uint32_t rf[2][4];
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            rf[kk][e] = pack_f16(rv[kk][e][0] * rsc[e & 1], rv[kk][e][1] * rsc[e & 1]);
                    // the table in two rounds of nine groups of 8 distances: a round's P loads
                    // are all issued before its first MMA, so the table waits for two L2 round
                    // trips (the first also covers r above), not one per group; while K/V
                    // streams saturate the memory system a round trip costs thousands of cycles.
                    // Each round's results set the steps of its part of the rows and are stored.
#pragma unroll
                    for (int rd = 0; rd < 2; ++rd) {
                        float res[kGrp][4];
                        uint32_t pb[kGrp][2][2];
#pragma unroll
                        for (int u = 0; u < kGrp; ++u)
#pragma unroll
                            for (int kk = 0; kk < 2; ++kk) {
                                pb[u][kk][0] = pack_f16(raw[u][kk].x, raw[u][kk].y);
                                pb[u][kk][1] = pack_f16(raw[u][kk].z, raw[u][kk].w);
                            }
                        bool finite = true;
#pragma unroll
                        for (int u = 0; u < kGrp; ++u) {
                            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int kk = 0; kk < 2; ++kk) mma_16816_f16(acc, rf[kk], pb[u][kk][0], pb[u][kk][1]);
                            res[u][0] = acc[0] * rusc[0];
                            res[u][1] = acc[1] * rusc[0];
                            res[u][2] = acc[2] * rusc[1];
                            res[u][3] = acc[3] * rusc[1];
                            finite = finite && isfinite(acc[0] + acc[1] + acc[2] + acc[3]);
                        }
                        if (!kCodes && rd == 0) ask(1);
                        // a P beyond fp16's range (|P| >= 65520) leaves an infinite or undefined entry
                        if (!finite) set_status(p.dev_status, INKATTN_ERR_DEVICE_BOUNDS);
                        // each token row's largest |entry| in this round (its four lanes hold all
                        // of its columns here)
                        float mx[2] = {0.f, 0.f};
#pragma unroll
                        for (int u = 0; u < kGrp; ++u) {
                            mx[0] = fmaxf(mx[0], fmaxf(fabsf(res[u][0]), fabsf(res[u][1])));
                            mx[1] = fmaxf(mx[1], fmaxf(fabsf(res[u][2]), fabsf(res[u][3])));
                        }
                        float enc[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
                            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
                            const float mm = fmaxf(mx[i], 1e-30f);
                            const int tt = gq + 8 * i;
                            // the step in S units (the table holds R / scale); entries encode to
                            // R * (32000 / max) in [-32000, 32000]
                            if (tq == 0 && tt < q_len) tsig[(hq * A.ql + tt) * 2 + rd] = mm * inv_scale * (1.f / 32000.f);
                            enc[i] = 32000.f / mm;
                        }
#pragma unroll
                        for (int u = 0; u < kGrp; ++u) {
                            const int c = (rd * kGrp + u) * 8 + 2 * tq;
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int tt = gq + 8 * i;
                                if (tt >= q_len) continue;
                                const float2 v = fix16_encode2(make_float2(res[u][2 * i], res[u][2 * i + 1]), enc[i]);
                                *reinterpret_cast<uint32_t *>(tab + ((size_t)hq * A.ql + tt) * kTabStride + c) =
                                    (__float_as_uint(v.x) & 0xFFFFu) | (__float_as_uint(v.y) << 16);
                            }
                        }
                        if (kCodes && rd == 0) ask(1);
                    }
                }
                mbar_arrive(bar(C::B_TAB_FULL));
                if (!(ok = wwait(bar(C::B_TAB_FULL), band_round & 1))) break;
            }

            if (!(ok = wwait(bar(C::B_S_FULL + (n & 1)), (n >> 1) & 1))) break;
            if (!quad_live) {
                // every row of this warp's lane quarter is padding: its P rows feed only O rows
                // that are never written, so the warp only keeps the barrier counts
                if (band) {
                    mbar_arrive(bar(C::B_TAB_FREE));
                    ++band_round;
                }
                tc::fence_before();
                if (!(A.withhold && n == 0)) mbar_arrive(bar(C::B_P_FULL + (n & 1)));
                continue;
            }
            tc::fence_after();
            const uint32_t sbuf = tmem + kTmemS0 + (uint32_t)(n & 1) * 128 + lane_off;
            float s[64];
            {
                uint32_t *su = reinterpret_cast<uint32_t *>(s);
                tc::ld32(sbuf + cb, *reinterpret_cast<uint32_t(*)[32]>(su));
                tc::ld32(sbuf + cb + 32, *reinterpret_cast<uint32_t(*)[32]>(su + 32));
                tc::wait_ld();
            }
            if (band) {
                if (valid_row) {
                    // column b of the tile is at distance i - j = dlo + (t + 127 - b)
                    const int c0 = t + (kKeys - 1) - cb;             // table column of key column cb
                    const unsigned short *trow = tab + ((size_t)hh * A.ql + t) * kTabStride + c0;
                    const float sg0 = tsig[(hh * A.ql + t) * 2], sg1 = tsig[(hh * A.ql + t) * 2 + 1];
                    const float sgm = hw == 0 ? sg1 : sg0;
#pragma unroll
                    for (int bb = 0; bb < 64; ++bb) {
                        const float q = __uint_as_float(0x4B000000u | (uint32_t)trow[-bb]) - 8421376.0f;
                        const bool mid = bb >= kTabMidLo && bb <= kTabMidHi;
                        s[bb] = fmaf(q, mid ? sgm : c0 - bb < 72 ? sg0 : sg1, s[bb]);
                    }
                }
                mbar_arrive(bar(C::B_TAB_FREE));
                ++band_round;
            }
            // mask: key j visible iff it is in this split's range, j <= i and (SWA) i - j < window
            int b_lo, span;
            {
                int jv_lo = kr_lo, jv_hi = min(i_pos, kr_hi - 1);
                if (p.window > 0) jv_lo = max(jv_lo, i_pos - p.window + 1);
                const bool any = valid_row && jv_hi >= jv_lo;
                b_lo = any ? jv_lo - j0 - cb : (1 << 20);
                span = any ? jv_hi - jv_lo : 0;
            }
            const bool need_mask = (!kCodes && !valid_row) || (j0 + kKeys - 1 > pos0) || (j0 + kKeys > kr_hi) ||
                                   (p.window > 0 && pos0 + q_len - 1 - j0 >= p.window);
            if (need_mask) {
#pragma unroll
                for (int bb = 0; bb < 64; ++bb)
                    s[bb] = ((unsigned)(bb - b_lo) <= (unsigned)span) ? s[bb] : -INFINITY;
            }
            float m4[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float m = fmax3(s[16 * c], s[16 * c + 1], s[16 * c + 2]);
#pragma unroll
                for (int e = 3; e < 15; e += 2) m = fmax3(m, s[16 * c + e], s[16 * c + e + 1]);
                m4[c] = fmaxf(m, s[16 * c + 15]);
            }
            float mx = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]);
            float *xc = xchg + (n & 1) * 256;
            xc[hw * 128 + a] = mx;
            pair_meet();
            ++met;
            mx = fmaxf(mx, xc[(1 - hw) * 128 + a]);
            const float mx_raw = mx;                             // the row's largest logit of the tile (S units)
            mx = mx == -INFINITY ? -INFINITY : mx * c_qk;        // log2 units
            const bool need = mx > m_run + 8.f;
            if (__any_sync(0xffffffffu, need)) {
                const float m_new = need ? fmaxf(m_run, mx) : m_run;
                const float corr = m_new == -INFINITY ? 1.f : fast_exp2(m_run - m_new);
                if (n > 0) {
                    if (!(ok = wait_pv(n - 1))) break;
                    tc::fence_after();
                    uint32_t o[32];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        tc::ld32(tmem + kTmemO + lane_off + cb + c * 32, o);
                        tc::wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                        tc::st32(tmem + kTmemO + lane_off + cb + c * 32, o);
                    }
                    tc::wait_st();
                }
                l_run *= corr;
                lc_run *= corr;
                m_run = m_new;
            }
            const float ref = m_run == -INFINITY ? 0.f : m_run;
            const float2 cq = make_float2(c_qk, c_qk), nref = make_float2(-ref, -ref);
            if (hw == 0 && mx_raw != -INFINITY) {
                // the tile's largest P of this row, computed as its element is, and its bf16 rounding
                const float pm = fast_exp2(fmaf(mx_raw, c_qk, -ref));
                if constexpr (kCodes) lc_run += __half2float(__float2half_rn(pm)) - pm;
                else lc_run += bf16_lo(pack_bf16(pm, 0.f)) - pm;
            }
            float2 l4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                            make_float2(0.f, 0.f)};
            uint32_t pk[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                const float2 x = ffma2(make_float2(s[2 * e], s[2 * e + 1]), cq, nref);
                const float2 y = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                l4[e & 3] = fadd2(l4[e & 3], y);
                pk[e] = kCodes ? pack_f16(y.x, y.y) : pack_bf16(y.x, y.y);
            }
            tc::st32(sbuf + 32 * hw, pk);
            const float2 l2 = fadd2(fadd2(l4[0], l4[1]), fadd2(l4[2], l4[3]));
            l_run += l2.x + l2.y;
            tc::wait_st();
            tc::fence_before();
            if (!(A.withhold && n == 0)) mbar_arrive(bar(C::B_P_FULL + (n & 1)));
        }
        // epilogue: the row sum of both halves, then O / l for this thread's 64 columns
        // the column-half 0 thread of a row alone holds the correction (lc_run is 0 in the other)
        // and alone writes the LSE: it publishes l + lc, the other thread l
        for (; met < N; ++met) pair_meet();
        float *xl = xchg + 512;
        xl[hw * 128 + a] = l_run + lc_run;
        pair_meet();
        const float l_other = xl[(1 - hw) * 128 + a];
        const float l_tot = l_run + l_other;                  // the fp32 sum (read by half 0 only)
        const float l_norm = l_run + lc_run + l_other;        // normaliser of P V's bf16 P
        if (ok) ok = wait_pv(N - 1);
        if (ok) {
            tc::fence_after();
            const float inv = l_norm > 0.f ? 1.f / l_norm : 0.f;
            const size_t qrow = (size_t)(start + t) * p.Hq + hk * g + hh;
            const float ref = m_run == -INFINITY ? 0.f : m_run;
            const float lse_nat = l_tot > 0.f ? (ref + log2f(l_tot)) * 0.6931471805599453f : -INFINITY;
            uint32_t o[32];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                tc::ld32(tmem + kTmemO + lane_off + cb + c * 32, o);
                tc::wait_ld();
                if (!valid_row) continue;
                const int col = cb + c * 32;
                if (A.S > 1) {
                    float4 *dst = reinterpret_cast<float4 *>(A.ws_o + (qrow * A.S + split) * kHeadDim + col);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dst[e] = make_float4(__uint_as_float(o[4 * e]) * inv, __uint_as_float(o[4 * e + 1]) * inv,
                                             __uint_as_float(o[4 * e + 2]) * inv, __uint_as_float(o[4 * e + 3]) * inv);
                } else if (p.out_dtype == INKATTN_DTYPE_F32) {
                    float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + qrow * kHeadDim + col);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dst[e] = make_float4(__uint_as_float(o[4 * e]) * inv, __uint_as_float(o[4 * e + 1]) * inv,
                                             __uint_as_float(o[4 * e + 2]) * inv, __uint_as_float(o[4 * e + 3]) * inv);
                } else {
                    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<inkattn_bf16 *>(p.out) + qrow * kHeadDim + col);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        dst[e] = make_uint4(
                            pack_bf16(__uint_as_float(o[8 * e]) * inv, __uint_as_float(o[8 * e + 1]) * inv),
                            pack_bf16(__uint_as_float(o[8 * e + 2]) * inv, __uint_as_float(o[8 * e + 3]) * inv),
                            pack_bf16(__uint_as_float(o[8 * e + 4]) * inv, __uint_as_float(o[8 * e + 5]) * inv),
                            pack_bf16(__uint_as_float(o[8 * e + 6]) * inv, __uint_as_float(o[8 * e + 7]) * inv));
                }
            }
            if (valid_row && hw == 0) {
                if (A.S > 1) A.ws_lse[qrow * A.S + split] = lse_nat;
                else if (p.lse) p.lse[qrow] = lse_nat;
            }
        }
    }

    tc::fence_before();
    __syncthreads();
    if (warp == C::kWarpMma) {
        tc::fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <int kKv>
cudaError_t launch_decode_variant(const DecTcArgs &a, dim3 grid, const CUtensorMap &qmap, const CUtensorMap &kmap,
                                  const CUtensorMap &vmap, cudaStream_t stream) {
    using C = Dec<kKv>;
    if constexpr (C::kCodes) {
        // the register split needs exactly kRegsLaunch registers a thread at launch: with fewer,
        // setmaxnreg.inc could never be satisfied
        static const cudaError_t regs_check = [] {
            cudaFuncAttributes fa;
            if (cudaFuncGetAttributes(&fa, k_decode_tc<kKv>) != cudaSuccess) return cudaErrorInvalidDeviceFunction;
            return fa.numRegs == C::kRegsLaunch ? cudaSuccess : cudaErrorInvalidConfiguration;
        }();
        if (regs_check != cudaSuccess) return regs_check;
    }
    cudaError_t err = cudaFuncSetAttribute(k_decode_tc<kKv>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (err != cudaSuccess) return err;
    return launch_dependent(k_decode_tc<kKv>, grid, dim3(C::kThreads), C::kSmem, stream, 1, a, qmap, kmap, vmap);
}

cudaError_t launch_decode_tc(const inkattn_attn_params &p, const AttnScalars &s, int num_splits,
                             float *ws_o, float *ws_lse, const CUtensorMap &qmap, const CUtensorMap &kmap,
                             const CUtensorMap &vmap, cudaStream_t stream) {
    DecTcArgs a;
    a.p = p;
    a.scale = s.scale;
    a.S = num_splits;
    a.band_split = num_splits == 2 && p.rel_extent > 0;
    a.ql = p.max_seqlen_q;
    a.ws_o = ws_o;
    a.ws_lse = ws_lse;
    a.kv_rows = (long long)p.num_blocks * p.Hkv * kBlock;
    a.wait_ns = kernel_debug().wait_ns;
    a.withhold = kernel_debug().withhold;
    a.i4_mask = kI4Mask;
    a.i4_exponent = kI4Exponent;
    const dim3 grid = a.band_split ? dim3(p.Hkv, p.B, 2) : dim3(num_splits, p.Hkv, p.B);
    switch (p.kv_dtype) {
        case INKATTN_KV_E4M3: return launch_decode_variant<INKATTN_KV_E4M3>(a, grid, qmap, kmap, vmap, stream);
        case INKATTN_KV_I4: return launch_decode_variant<INKATTN_KV_I4>(a, grid, qmap, kmap, vmap, stream);
        default: return launch_decode_variant<INKATTN_KV_BF16>(a, grid, qmap, kmap, vmap, stream);
    }
}

}  // namespace inkattn
