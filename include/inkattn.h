/*
 * inkattn.h -- C ABI of libinkattn.so, the GB300 (sm_103a) attention hot path of
 * one Inkling decoder layer, the layer's products behind it, and the end of a
 * verification step.
 *
 * Sources, cited by page title and section heading:
 *   [SG] "SGLang と Miles が Inkling を初日からサポート：975Bのマルチモーダル最先端モデルが公開"
 *        (winzheng.jp review page)
 *   [VJ] "vLLM TML Inkling サポート" (agentlenshq.com, Japanese)
 *   [VV] "vLLM hỗ trợ TML Inkling ngay khi ra mắt với hiệu năng tối ưu" (gpuhub.net)
 *
 * General conventions
 *   - Every pointer inside a params struct is a DEVICE pointer owned by the caller.
 *     The library allocates no device memory at run time: the split-KV partials of
 *     inkattn_decode live in a caller-provided workspace, those of
 *     inkattn_decode_noalloc in a fixed 64 MiB buffer that is part of the library image.
 *   - bf16 tensors are IEEE bfloat16 (inkattn_bf16 holds the raw 16-bit pattern);
 *     all arrays are dense and row-major in the layouts stated per field.
 *   - Every call is asynchronous on the caller's CUDA stream (passed as void*, a
 *     cudaStream_t; NULL = the legacy default stream), keeps no state between calls
 *     and is safe to call from several host threads.
 *   - Kernels are chained by programmatic dependent launch: each may become resident on
 *     the GPU while the kernel before it on the stream finishes, and reads no global
 *     memory before that kernel has completed, so stream order holds as for any launch.
 *     inkattn_prologue, inkattn_output_conv, inkattn_qkvr_prologue, the calls of the layer's
 *     second half and those of a verification step's end let the next kernel be scheduled once all their CTAs have
 *     started; the attention kernels do not.  Every call can be captured
 *     into a CUDA graph.
 *   - Host-side validation runs before any launch; on failure the call returns
 *     INKATTN_ERR_INVALID_ARG or INKATTN_ERR_UNSUPPORTED and launches nothing.
 *   - Alignment: bf16 arrays (activations, caches, conv states, outputs) must be 16-byte
 *     aligned; the fp32 conv weights and RMSNorm gains of inkattn_prologue and
 *     inkattn_qkvr_prologue, the index arrays, lse and dev_status 4-byte aligned; further
 *     rules are stated per entry point.  A pointer that breaks its rule is
 *     INKATTN_ERR_INVALID_ARG.
 *   - Index arrays are read only on the device.  Kernels bounds-check every index
 *     they read (cu_seqlens_q, seqlen_k, state_slot, slot_mapping, block_table);
 *     an out-of-range value skips the access and, when dev_status is non-NULL,
 *     writes INKATTN_ERR_DEVICE_BOUNDS there.  Bounded device waits that run out
 *     write INKATTN_ERR_DEVICE_TIMEOUT.  The first error written wins; the caller
 *     zeroes *dev_status before the call and reads it after synchronising.
 *   - head_dim must be 128 and block_size 64, else INKATTN_ERR_UNSUPPORTED.
 *   - Bounded device waits give up after 1 s.  For tests of that failure path only, two
 *     environment variables are read once per process: INKATTN_TEST_WAIT_LIMIT_US
 *     (100 .. 10000000: a shorter limit) and INKATTN_TEST_WITHHOLD_ARRIVAL=1 (the
 *     attention kernels' softmax withholds its first arrival before P V, and the qkvr and
 *     linear kernels one release of an accumulator, so that the MMA warp's wait runs out).  Leave
 *     both unset in normal use.
 */
#ifndef INKATTN_H
#define INKATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define INKATTN_ABI_VERSION 2

/* The library is built with hidden visibility; only these entry points are exported. */
#if defined(__GNUC__)
#define INKATTN_API __attribute__((visibility("default")))
#else
#define INKATTN_API
#endif

typedef uint16_t inkattn_bf16;

/* Element type of the attention output. */
#define INKATTN_DTYPE_BF16 0
#define INKATTN_DTYPE_F32 1

/* Element type of the paged KV cache (kv_dtype).
 * INKATTN_KV_BF16: k_cache and v_cache hold bf16 values.
 * INKATTN_KV_E4M3: they hold OCP FP8 E4M3 codes (1 byte per value, same
 *   [num_blocks][Hkv][64][128] layout), and k_scale / v_scale hold one fp32 scale per
 *   row ([num_blocks][Hkv][64]): the row's values are code * scale.  The prologue writes
 *   scale = 2^k, k the smallest integer >= -24 with 448 * 2^k >= the row's largest
 *   magnitude (1 for an all-zero row), and each code as the nearest E4M3 value to
 *   x / 2^k (ties to even), where x is the bf16 value the bf16 cache would hold; the
 *   dequantised value is exact.  [SG §Relative Attention と FA4 経路: MXFP8 on the FA4
 *   path; VJ §フューチャーロードマップ and VV: FP8 for the global-attention layers.]
 *   The decode reads such a cache, and inkattn_prefill_e4m3 (inkattn_prefill returns
 *   INKATTN_ERR_UNSUPPORTED for it).
 *   The decode expands each row to f16 (code * scale, exact for the prologue's scales
 *   down to 2^-15; below, values under 2^-24 flush) and requires every scale to lie in
 *   [2^-24, 2^7], which the prologue's scales do for rows whose magnitudes stay below
 *   57344; a scale outside that range is flagged as INKATTN_ERR_DEVICE_BOUNDS and its
 *   row read as zeros.
 * INKATTN_KV_I4: they hold 4-bit whole numbers, [num_blocks][Hkv][64] rows of 64 bytes (128
 *   values), and k_scale / v_scale, passed through the same pointers, hold 4 scale bytes per
 *   row ([num_blocks][Hkv][64][4] uint8), one per group of 32 values.  A scale byte b stands
 *   for s = the fp16 of bits b << 7 (5 exponent and 3 mantissa bits), 0 .. 896 (b <= 0xC6).
 *   Little-endian 32-bit word w of a row holds its values 8 w .. 8 w + 7 as u = n + 8, n in
 *   [-7, 7], value 8 w + 2 i in bits 4 i .. 4 i + 3 and value 8 w + 2 i + 1 in bits 16 + 4 i
 *   .. 19 + 4 i; a value reads back as n * s, exact in bf16.  The prologue writes the smallest
 *   s with 7 s >= the group's largest magnitude (0 for a zero group, 896 at most, beyond which
 *   values saturate at 7 * 896 = 6272), and n = x / s rounded to nearest, ties to even, where x is the
 *   bf16 value the bf16 cache would hold (a NaN is stored as 0).  Its caches are read by
 *   inkattn_decode and inkattn_prefill_i4 (inkattn_prefill returns INKATTN_ERR_UNSUPPORTED).  A
 *   scale byte above 0xC6 inside a sequence is flagged as INKATTN_ERR_DEVICE_BOUNDS and its group
 *   read as zeros; u = 0 is no code of the prologue's (it reads as -8 s).
 * Over a cache of codes (E4M3, I4) the decode holds q as fp16: |q| <= 65280; a value beyond that, or a NaN, is
 *   flagged as INKATTN_ERR_DEVICE_BOUNDS and its row's result undefined; below 2^-14 values count in steps of 2^-24. */
#define INKATTN_KV_BF16 0
#define INKATTN_KV_E4M3 1
#define INKATTN_KV_I4 4

typedef enum inkattn_status {
    INKATTN_OK = 0,
    INKATTN_ERR_INVALID_ARG = 1,     /* bad pointer, size, or combination of sizes     */
    INKATTN_ERR_UNSUPPORTED = 2,     /* valid but not implemented (head_dim, block ...) */
    INKATTN_ERR_CUDA = 3,            /* a CUDA runtime call or launch failed            */
    INKATTN_ERR_DEVICE_TIMEOUT = 4,  /* written to *dev_status by a bounded device wait */
    INKATTN_ERR_DEVICE_BOUNDS = 5    /* written to *dev_status by a device bounds check */
} inkattn_status;

/* Short English text for a status code (static storage, never NULL). */
INKATTN_API const char *inkattn_status_string(inkattn_status s);

/* INKATTN_ABI_VERSION of the built library. */
INKATTN_API int inkattn_abi_version(void);

/* ------------------------------------------------------------------------------
 * The attention prologue [SG §ShortConv 最適化：融合、グラフキャプチャ、シャーディング]:
 * K/V ShortConv + conv-state carry + Q/K RMSNorm + paged KV write, one kernel.
 *
 * Let C = Hkv*128, g = Hq/Hkv.  Sequence b owns new tokens
 * [cu_seqlens_q[b], cu_seqlens_q[b+1]).  For each sequence and channel c, with xs =
 * the 3 carried rows (oldest first) followed by the new rows of k (resp. v):
 *   kc[t][c] = bf16( sum_{k=0..3} conv_w_k[c][k] * xs[t+k][c] )     (fp32 accumulate,
 *   vc[t][c] = bf16( same with v and conv_w_v )                      taps in order 0..3)
 * [SG §ShortConv：4カ所に現れる短距離因果畳み込み: W = 4, current token plus the 3 previous
 * positions of the same channel; conv_w[c][3] weighs the current token].
 * The state slot then holds the last 3 rows of xs [VV §Quản lý bộ nhớ đệm sconv].
 * Per (token, head) over the 128 values, in fp32, rounded to bf16:
 *   q_out = q  / sqrt(mean(q^2)  + eps) * q_norm_w
 *   kn    = kc / sqrt(mean(kc^2) + eps) * k_norm_w
 * [SG §Inkling のモデルアーキテクチャ: ShortConv on K and V before the Q/K normalisation].
 * Then, with slot = slot_mapping[t]: k_cache[slot/64][hk][slot%64][:] = kn,
 * v_cache[...] = vc (with kv_dtype = INKATTN_KV_E4M3 or INKATTN_KV_I4: their codes, and the
 * scales to k_scale / v_scale[slot/64][hk][slot%64]).  V is not normalised and Q is not
 * convolved.
 * ------------------------------------------------------------------------------ */
typedef struct inkattn_prologue_params {
    size_t struct_size;        /* = sizeof(inkattn_prologue_params)                      */
    int32_t B;                 /* sequences in the batch, >= 1                           */
    int32_t N_tok;             /* new tokens = cu_seqlens_q[B], >= 0                     */
    int32_t max_seqlen_q;      /* >= every q_len[b]; sizes the grid                      */
    int32_t Hq, Hkv;           /* query / KV heads, Hq % Hkv == 0                        */
    int32_t head_dim;          /* 128                                                    */
    int32_t block_size;        /* paged-cache block, 64                                  */
    int32_t num_blocks;        /* cache capacity in blocks (bounds check)                */
    int32_t num_state_slots;   /* conv-state capacity in slots (bounds check)            */
    float eps;                 /* RMSNorm epsilon, >= 0                                  */
    const inkattn_bf16 *q;     /* [N_tok][Hq][128]                                       */
    const inkattn_bf16 *k;     /* [N_tok][C]  (K projection output, before the conv)     */
    const inkattn_bf16 *v;     /* [N_tok][C]                                             */
    const float *conv_w_k;     /* [C][4]                                                 */
    const float *conv_w_v;     /* [C][4]                                                 */
    const float *q_norm_w;     /* [128], shared by all query heads                       */
    const float *k_norm_w;     /* [128], shared by all KV heads                          */
    const int32_t *cu_seqlens_q;   /* [B+1], non-decreasing, cu[0] = 0                   */
    const int32_t *state_slot;     /* [B], distinct values in [0, num_state_slots)       */
    const int32_t *slot_mapping;   /* [N_tok], distinct values in [0, num_blocks*64)     */
    inkattn_bf16 *conv_state_k;    /* [num_state_slots][3][C], read then overwritten     */
    inkattn_bf16 *conv_state_v;    /* [num_state_slots][3][C]                            */
    inkattn_bf16 *q_out;           /* [N_tok][Hq][128]                                   */
    void *k_cache;                 /* [num_blocks][Hkv][64][128], bf16, E4M3 or 4 bits (kv_dtype) */
    void *v_cache;                 /* [num_blocks][Hkv][64][128]                         */
    int32_t kv_dtype;              /* INKATTN_KV_BF16 (0), INKATTN_KV_E4M3 (1) or INKATTN_KV_I4 (4) */
    float *k_scale;                /* E4M3: [num_blocks][Hkv][64] row scales; I4: 4 scale bytes a row; */
    float *v_scale;                /* 16-byte aligned; written for the mapped slots (bf16: NULL) */
    int32_t *dev_status;           /* nullable, see the conventions above                */
} inkattn_prologue_params;

/* Runs the prologue.  Buffers may not alias except as stated (conv_state_* in/out). */
INKATTN_API inkattn_status inkattn_prologue(const inkattn_prologue_params *p, void *stream);

/* ------------------------------------------------------------------------------
 * Relative-position-bias GQA attention over the paged cache
 * [SG §相対位置バイアス付き Attention; VJ §TML Inkling モデルアーキテクチャ
 *  "Hybrid Attention", "Relative Attention"; VV §FA4 với sheared bias].
 *
 * Sequence b has q_len = cu_seqlens_q[b+1]-cu_seqlens_q[b] new tokens at positions
 * i = seqlen_k[b]-q_len+t; key j (0 <= j < seqlen_k[b]) sits at position j in block
 * block_table[b][j/64], offset j%64, head kv = h / (Hq/Hkv).  For query head h:
 *   s_ij = lambda_b * ( softmax_scale * q_i.k_j + bias_hij ),
 *   bias_hij = sum_{e<d_r} r[i][h][e] * P[h][i-j][e]  if 0 <= i-j < rel_extent, else 0,
 * visible keys: j <= i, and i-j < window when window > 0 (sliding-window layer),
 *   lambda_b = max(1, ln(seqlen_k[b]) / ln(log_scale_base)) when log_scale_base > 1
 *             (full layers' length-dependent logit scaling), else 1,
 *   out_i = sum_j softmax_j(s_ij) v_j,  lse_i = ln sum_j exp(s_ij)  (natural log).
 * softmax_scale <= 0 selects 1/sqrt(128).
 *
 * q, k_cache and v_cache are read by TMA through tensor maps and must be device memory of
 * the current device (cudaMalloc or a memory pool of that device); host memory, managed
 * memory and another GPU's memory are rejected with INKATTN_ERR_INVALID_ARG.  The prefill
 * kernel multicasts each K/V tile to the two CTAs of a head pair inside one cluster: the
 * tensor maps cover this GPU's memory alone.
 * The bias enters the logits as 16-bit fixed point in units of softmax_scale * q.k, so the
 * absolute error of a bias value is at most half a step.  Prefill takes one step per chunk
 * of 128 distances, max_a |r_a| * max_delta |P_h[delta]| / 32000 over the chunk's rows and
 * distances (by Cauchy-Schwarz no value of the chunk exceeds 32000 steps); decode takes one
 * per query row and table round, the largest magnitude in it / 32000.  The
 * decode tables are computed with fp16 operands: P's entries must lie inside fp16's range
 * (|P| < 65504), else the call reports INKATTN_ERR_DEVICE_BOUNDS.
 * ------------------------------------------------------------------------------ */
typedef struct inkattn_attn_params {
    size_t struct_size;        /* = sizeof(inkattn_attn_params)                          */
    int32_t B;                 /* sequences, >= 1                                        */
    int32_t N_tok;             /* query rows = cu_seqlens_q[B]                           */
    int32_t max_seqlen_q;      /* >= every q_len[b]                                      */
    int32_t max_seqlen_k;      /* >= every seqlen_k[b]                                   */
    int32_t Hq, Hkv;           /* Hq % Hkv == 0                                          */
    int32_t head_dim;          /* 128                                                    */
    int32_t block_size;        /* 64                                                     */
    int32_t num_blocks;        /* cache capacity in blocks (bounds check)                */
    int32_t max_blocks_per_seq;/* row length of block_table                              */
    int32_t d_r;               /* relative feature size: 32                              */
    int32_t rel_extent;        /* >= 0; 0 disables the bias                              */
    int32_t window;            /* 0 = full attention, else the sliding window (keys)     */
    int32_t out_dtype;         /* INKATTN_DTYPE_BF16 (0) or INKATTN_DTYPE_F32 (1) for out */
    float softmax_scale;       /* <= 0 -> 1/sqrt(128)                                    */
    float log_scale_base;      /* <= 1 -> no length-dependent scaling (8192 on full layers) */
    const inkattn_bf16 *q;     /* [N_tok][Hq][128], the normalised queries               */
    const inkattn_bf16 *r;     /* [N_tok][Hq][d_r], 16-byte aligned (nullable iff rel_extent == 0) */
    const float *P;            /* [Hq][rel_extent][d_r]: per query head, per distance,   */
                               /* the d_r projection weights; 16-byte aligned (nullable  */
                               /* iff rel_extent == 0)                                   */
    const void *k_cache;           /* [num_blocks][Hkv][64][128], bf16, E4M3 or 4 bits (kv_dtype) */
    const void *v_cache;           /* [num_blocks][Hkv][64][128]                         */
    int32_t kv_dtype;              /* INKATTN_KV_BF16 (0), INKATTN_KV_E4M3 (1) or INKATTN_KV_I4 (4) */
    const float *k_scale;          /* E4M3: [num_blocks][Hkv][64] row scales; I4: 4 scale bytes a row; */
    const float *v_scale;          /* 16-byte aligned (bf16: NULL)                       */
    const int32_t *cu_seqlens_q;   /* [B+1]                                              */
    const int32_t *seqlen_k;       /* [B], q_len[b] <= seqlen_k[b] <= max_seqlen_k       */
    const int32_t *block_table;    /* [B][max_blocks_per_seq]                            */
    void *out;                     /* [N_tok][Hq][128], bf16 or fp32 per out_dtype; the   */
                                   /* bf16 form is the fp32 result rounded once (RNE)     */
    float *lse;                    /* nullable, [N_tok][Hq]                              */
    int32_t *dev_status;           /* nullable                                           */
} inkattn_attn_params;

/* Prefill (any q_len) over a bf16 cache: writes out (and lse).  An E4M3 or 4-bit cache returns
 * INKATTN_ERR_UNSUPPORTED here; it takes inkattn_prefill_e4m3 or inkattn_prefill_i4. */
INKATTN_API inkattn_status inkattn_prefill(const inkattn_attn_params *p, void *stream);

/* Prefill over an E4M3 cache (kv_dtype = INKATTN_KV_E4M3) [SG §Relative Attention と FA4
 * 経路; VJ §フューチャーロードマップ: FP8 for the global-attention layers].  The blocks the
 * batch reads, block_table[b][0 .. ceil(seqlen_k[b]/64)), are first expanded, code * scale
 * (exact in bf16), into a bf16 copy in the workspace with a block table of its own; then the
 * bf16 prefill runs on the copy, so the result is the bf16 prefill's over the dequantised
 * cache.  A row inside a sequence whose scale lies outside [2^-24, 2^7] (or a block id out
 * of range) is flagged INKATTN_ERR_DEVICE_BOUNDS and read as zeros, as in the decode.
 * workspace: device memory of the current device, 256-byte aligned, at least
 * inkattn_prefill_workspace_bytes(p) bytes (B * max_blocks_per_seq blocks of bf16 K and V
 * plus their table), else INKATTN_ERR_INVALID_ARG; a bf16 cache is INKATTN_ERR_INVALID_ARG
 * (it takes inkattn_prefill).  Two launches, chained like the others. */
INKATTN_API size_t inkattn_prefill_workspace_bytes(const inkattn_attn_params *p);   /* 0 if invalid or bf16 */
INKATTN_API inkattn_status inkattn_prefill_e4m3(const inkattn_attn_params *p, void *workspace,
                                                size_t workspace_bytes, void *stream);

/* The same over a 4-bit cache (kv_dtype = INKATTN_KV_I4; a bf16 or E4M3 one is
 * INKATTN_ERR_INVALID_ARG): same workspace, its size from inkattn_prefill_workspace_bytes,
 * n * s exact in the bf16 copy, a group with a scale byte above 0xC6 flagged and read as zeros. */
INKATTN_API inkattn_status inkattn_prefill_i4(const inkattn_attn_params *p, void *workspace, size_t workspace_bytes,
                                              void *stream);

/* ------------------------------------------------------------------------------
 * Split-KV decode [VJ §低レイテンシコレクティブとカーネル "FA4 Kernel"; VV §FA4 với
 * sheared bias: num_splits is picked per configuration from batch size, TP size and
 * KV length].  Decode shapes: max_seqlen_q <= 16 and max_seqlen_q*(Hq/Hkv) <= 128
 * (e.g. 9 MTP-verify tokens x 8 query heads per KV head).  Same math as prefill.
 * ------------------------------------------------------------------------------ */

/* The split count the library would pick for these params on a GPU with num_sms
 * SMs (tensor-parallel size 1).  Host only; returns >= 1, or 0 for invalid params. */
INKATTN_API int inkattn_decode_num_splits(const inkattn_attn_params *p, int num_sms);

/* Bytes of workspace inkattn_decode needs for num_splits (0 = the heuristic on the
 * current device): N_tok*Hq*S*(128+1)*4 rounded up to 256, or 0 when S resolves to 1. */
INKATTN_API size_t inkattn_decode_workspace_bytes(const inkattn_attn_params *p, int num_splits);

/* Decode pass.  num_splits: 0 = heuristic, else 1..64.  The keys a sequence attends to
 * are divided into num_splits contiguous parts of near-equal size, except that with
 * num_splits = 2 and rel_extent > 0 the cut is at the start of the band (the keys
 * within rel_extent of the first query, moved down so that the part before it holds
 * whole 128-key tiles): the
 * streaming part and the band part then run in separate CTAs, the streaming ones
 * scheduled first.  Over a 4-bit cache the other split counts divide the keys into parts of about equal
 * cost instead, whole 128-key tiles, a tile of the band counting for several others.  With one split the result goes straight to out/lse; otherwise each
 * split's own softmax-normalised partial output and its lse go to the workspace, and
 * inkattn_combine must follow on the same stream with the same num_splits.
 * workspace: device memory of at least inkattn_decode_workspace_bytes bytes,
 * 256-byte aligned, owned by the caller, not read by the host. */
INKATTN_API inkattn_status inkattn_decode(const inkattn_attn_params *p, int num_splits,
                              void *workspace, size_t workspace_bytes, void *stream);

/* Merges the per-split partials: lse = ln sum_s exp(lse_s), out = sum_s
 * exp(lse_s - lse) out_s.  A no-op when num_splits resolves to 1. */
INKATTN_API inkattn_status inkattn_combine(const inkattn_attn_params *p, int num_splits,
                               const void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------------
 * Decode without a caller-provided workspace.  The pages have no counterpart: this
 * is a library convenience.
 *
 * For callers that cannot allocate device memory where they decode: plugin hosts that
 * own all device memory and pass only inputs and outputs, and serving loops that must not
 * allocate on the hot path (an allocation can synchronise the device).  The call itself
 * still makes CUDA runtime calls (device and pointer queries, tensor-map encoding) and
 * launches kernels.
 *
 * Same computation and result as inkattn_decode followed by inkattn_combine with the
 * same split count, writing out/lse: with an explicit num_splits the results are
 * bit-identical to theirs.  The split partials go to a static device buffer of
 * INKATTN_DECODE_NOALLOC_MAX_BYTES inside the library instead of a workspace; the call
 * allocates nothing (no cudaMalloc, cudaFree or allocating library routine).
 *   - num_splits = 0 takes the heuristic's split count and lowers it until the partials
 *     fit the buffer (down to 1, which needs none).
 *   - An explicit num_splits whose partials exceed the buffer, i.e. whose
 *     inkattn_decode_workspace_bytes(p, S) is above INKATTN_DECODE_NOALLOC_MAX_BYTES, is
 *     rejected with INKATTN_ERR_INVALID_ARG.
 *   - The buffer's device address belongs to a CUDA context; it is looked up with the
 *     caller's context current and cached per context (a new context, e.g. after
 *     cudaDeviceReset, looks it up again).  The first call in a context may load the
 *     library's device code: make it before any stream capture.
 *   - Every call on a device shares the one buffer and it keeps the last call's
 *     contents.  Each call writes every partial it reads, so nothing needs clearing,
 *     but calls whose GPU work overlaps (on different streams, or from several host
 *     threads without ordering) race on the buffer: serialise them.
 *   - Each GPU on which this part of the library is loaded holds the buffer until the
 *     process exits.
 * ------------------------------------------------------------------------------ */
#define INKATTN_DECODE_NOALLOC_MAX_BYTES (64u << 20)

INKATTN_API inkattn_status inkattn_decode_noalloc(const inkattn_attn_params *p, int num_splits,
                                                  void *stream);

/* ------------------------------------------------------------------------------
 * Attention-output ShortConv with the residual add and the RMSNorm, one kernel
 * [SG §ShortConv：4カ所に現れる短距離因果畳み込み (the third ShortConv position, after the
 * attention output); SG §ShortConv 最適化：融合、グラフキャプチャ、シャーディング (it sits on the
 * residual stream; in decode the residual add and the RMSNorm fold into the same
 * kernel); VV §TP sharding nhận biết sconv (order: o_proj output -> sconv -> residual
 * connection -> RMSNorm)].  On one GPU there is no all-reduce in front of it: the input is
 * the o_proj output itself.
 *
 * For each sequence b and hidden channel c, with xs = the 3 carried rows (oldest first)
 * followed by the new rows of y:
 *   conv[t][c] = bf16( sum_{k=0..3} conv_w[c][k] * xs[t+k][c] )   (correctly rounded)
 *   h[t][c]    = bf16( residual[t][c] + conv[t][c] )               (correctly rounded)
 *   out[t][c]  = bf16( h[t][c] / sqrt(mean_c'(h[t][c']^2) + eps) * norm_w[c] )
 * the mean over all D channels of the token.  The state slot then holds the last 3 rows
 * of xs.  conv and h are bit-exact; out is within 1 bf16 ulp of the fp64 value (its sum
 * of squares is taken in fp32).  An empty sequence keeps its state.
 * ------------------------------------------------------------------------------ */
typedef struct inkattn_output_conv_params {
    size_t struct_size;        /* = sizeof(inkattn_output_conv_params)                   */
    int32_t B;                 /* sequences, 1 .. 65535                                  */
    int32_t N_tok;             /* new tokens = cu_seqlens_q[B], >= 0                     */
    int32_t max_seqlen_q;      /* >= every q_len[b]; sizes the grid                      */
    int32_t D;                 /* hidden width: a multiple of 8, 8 .. 32768              */
    int32_t num_state_slots;   /* conv-state capacity in slots (bounds check)            */
    float eps;                 /* RMSNorm epsilon, >= 0                                  */
    const inkattn_bf16 *y;     /* [N_tok][D], the o_proj output                          */
    const float *conv_w;       /* [D][4], w[c][3] weighs the current token               */
    const float *norm_w;       /* [D]                                                    */
    const int32_t *cu_seqlens_q;   /* [B+1], non-decreasing, cu[0] = 0                   */
    const int32_t *state_slot;     /* [B], distinct values in [0, num_state_slots)       */
    inkattn_bf16 *conv_state;      /* [num_state_slots][3][D], read then overwritten     */
    const inkattn_bf16 *residual;  /* [N_tok][D], the residual stream before the add     */
    inkattn_bf16 *h_out;           /* [N_tok][D], the new residual stream; may equal residual */
    inkattn_bf16 *out;             /* [N_tok][D], its RMSNorm                            */
    int32_t *dev_status;           /* nullable, see the conventions above                */
} inkattn_output_conv_params;

/* Runs the attention-output conv.  y, conv_w, norm_w, conv_state, residual, h_out and out
 * must be 16-byte aligned.  out and h_out may not overlap y, and out may not overlap
 * residual or h_out (INKATTN_ERR_INVALID_ARG); h_out == residual (in place) is allowed,
 * a partial overlap of the two is not.  conv_state must not overlap the other arrays. */
INKATTN_API inkattn_status inkattn_output_conv(const inkattn_output_conv_params *p, void *stream);

/* ------------------------------------------------------------------------------
 * The qkvr projections with the attention prologue fused into their epilogue: one pass
 * from the hidden states to what inkattn_prologue writes, plus r
 * [VJ §TML Inkling モデルアーキテクチャ and VV, the MoE item of the architecture list: the
 * q, k, v and r projections ("qkvr linears") are one bf16 linear layer in front of the
 * attention; SG §ShortConv 最適化：融合、グラフキャプチャ、シャーディング: the prologue's work
 * fused so that nothing intermediate is written back].
 *
 * With F = Hq*128 + 2*Hkv*128 + Hq*d_r output features and the rows of w ordered
 * [q heads | k | v | r heads] (nn.Linear layout, [F][d_model]):
 *   y[t][o] = bf16( sum_k x[t][k] * w[o][k] )       (fp32 accumulation on the tensor cores)
 *   q = y[:, 0:Hq*128] as [N_tok][Hq][128],  k = the next Hkv*128 features,
 *   v = the next Hkv*128,  r = the last Hq*d_r as [N_tok][Hq][d_r] (written to r_out).
 * Then everything inkattn_prologue does, on q, k and v, with two differences: the conv
 * state is read from conv_state_*_in and the new state written to conv_state_*_out, and
 * a sequence with no new tokens copies its state from in to out.  The projections are
 * rounded once from the fp32 sum; against the exactly rounded sum that can differ by one
 * bf16 ulp where the sum lies within the fp32 accumulation error of a rounding midpoint.
 *
 * Work is cut into tiles of INKATTN_QKVR_TILE_TOKENS (125) new tokens of one sequence plus
 * the 3 before them (the conv's history, recomputed rather than exchanged), so a tile
 * never waits on another.  The new conv state is written by the tile holding a sequence's
 * last tokens while the sequence's first tile reads the old one; in and out may therefore
 * be the same array only when max_seqlen_q <= INKATTN_QKVR_TILE_TOKENS (every sequence in
 * one tile), else INKATTN_ERR_INVALID_ARG.
 * ------------------------------------------------------------------------------ */
#define INKATTN_QKVR_TILE_TOKENS 125
#define INKATTN_QKVR_MAX_SEQS 1024

typedef struct inkattn_qkvr_params {
    size_t struct_size;        /* = sizeof(inkattn_qkvr_params)                          */
    int32_t B;                 /* sequences, 1 .. INKATTN_QKVR_MAX_SEQS                  */
    int32_t N_tok;             /* new tokens = cu_seqlens_q[B], >= 0                     */
    int32_t max_seqlen_q;      /* >= every q_len[b]                                      */
    int32_t Hq, Hkv;           /* query / KV heads, Hq % Hkv == 0                        */
    int32_t head_dim;          /* 128                                                    */
    int32_t d_r;               /* relative features per query head; Hq*d_r % 8 == 0      */
    int32_t d_model;           /* hidden width: a multiple of 8, >= 8                    */
    int32_t block_size;        /* paged-cache block, 64                                  */
    int32_t num_blocks;        /* cache capacity in blocks (bounds check)                */
    int32_t num_state_slots;   /* conv-state capacity in slots (bounds check)            */
    float eps;                 /* RMSNorm epsilon, >= 0                                  */
    const inkattn_bf16 *x;     /* [N_tok][d_model] hidden states; device memory of this GPU */
    const inkattn_bf16 *w;     /* [F][d_model]; device memory of this GPU                */
    const float *conv_w_k;     /* [C][4], C = Hkv*128; w[c][3] weighs the current token  */
    const float *conv_w_v;     /* [C][4]                                                 */
    const float *q_norm_w;     /* [128]                                                  */
    const float *k_norm_w;     /* [128]                                                  */
    const int32_t *cu_seqlens_q;   /* [B+1], non-decreasing, cu[0] = 0                   */
    const int32_t *state_slot;     /* [B], distinct values in [0, num_state_slots)       */
    const int32_t *slot_mapping;   /* [N_tok], distinct values in [0, num_blocks*64)     */
    const inkattn_bf16 *conv_state_k_in;  /* [num_state_slots][3][C]                     */
    const inkattn_bf16 *conv_state_v_in;  /* [num_state_slots][3][C]                     */
    inkattn_bf16 *conv_state_k_out;       /* [num_state_slots][3][C], rows of the        */
    inkattn_bf16 *conv_state_v_out;       /* sequences' slots written                    */
    inkattn_bf16 *q_out;           /* [N_tok][Hq][128], normalised                       */
    inkattn_bf16 *r_out;           /* [N_tok][Hq][d_r]                                   */
    inkattn_bf16 *y_out;           /* nullable: [N_tok][F], every projection as rounded  */
    void *k_cache;                 /* as in inkattn_prologue_params                      */
    void *v_cache;
    int32_t kv_dtype;              /* INKATTN_KV_BF16, INKATTN_KV_E4M3 or INKATTN_KV_I4   */
    float *k_scale;                /* scales of a cache of codes (else NULL), as in inkattn_prologue_params */
    float *v_scale;
    int32_t *dev_status;           /* nullable, see the conventions above                */
} inkattn_qkvr_params;

/* Runs the fused projections and prologue.  x and w are read by TMA (device memory of the
 * current device, 16-byte aligned; anything else is INKATTN_ERR_INVALID_ARG); q_out,
 * r_out, y_out, the caches and the states must be 16-byte aligned.  With y_out non-NULL the
 * projections (before conv and norm) are written there too, at the cost of their bytes.  No output may overlap an
 * input except conv_state_*_out == conv_state_*_in under the rule above. */
INKATTN_API inkattn_status inkattn_qkvr_prologue(const inkattn_qkvr_params *p, void *stream);

/* ------------------------------------------------------------------------------
 * The rest of the decoder layer.  Between the attention and inkattn_output_conv sits the
 * output projection [VV §TP sharding nhận biết sconv: o_proj output -> sconv -> residual
 * connection -> RMSNorm]; after it comes the MoE [SG §Inkling のモデルアーキテクチャ: sigmoid
 * scores, the 6 best of 256 routed experts, 2 shared experts that join the normalisation of
 * the weights but not the choice], whose output goes through the layer's fourth ShortConv
 * (inkattn_output_conv again).  inkattn_linear, inkattn_route, inkattn_grouped_linear and
 * inkattn_expert_combine are those products and what lies between them.
 *
 * The two products accumulate in fp32, apply bias and activation to the fp32 sums, and round
 * once to the output type.  They run on the tensor cores, except linear layers of few tokens or
 * of a small size, which are summed by fp32 multiply-adds.  The tensor cores do not round their
 * sums to nearest: fp32 outputs are therefore summed in parts of K = 512 (5e-7 of the result at
 * K = 8192), bf16 outputs in one (1e-5 at K = 8192, before a rounding of up to 4e-3).  With
 * v = x w^T + bias:
 *   NONE v   RELU max(v, 0)   GELU v (1 + erf(v / sqrt 2)) / 2   SILU v / (1 + exp(-v))
 *   (a NaN stays a NaN; an infinite v as in the formula, so that GELU and SILU of -infinity are
 *   NaN.  fp32 outputs: SILU within 11 units of 2^-24 of the value, GELU within 18, and 1.25 v^2
 *   more for negative v; values below 2^-126 within 2^-141.  bf16 outputs, before their
 *   rounding: GELU within 1.5e-7 |v| / 2, SILU within (4 + 1.2 |v|) 2^-23 of the value and 0
 *   below 2^-126)
 *   SWIGLU   w (and bias) hold 2 F rows, F gate rows first, then F up rows:
 *            SILU(gate) * up, F values.
 * Results do not depend on the GPU's scheduling: every sum is added in a fixed order.
 * In these four calls an array without rows (N_tok == 0, M == 0) may be NULL.
 * ------------------------------------------------------------------------------ */
#define INKATTN_ACT_NONE 0
#define INKATTN_ACT_RELU 1
#define INKATTN_ACT_GELU 2
#define INKATTN_ACT_SILU 3
#define INKATTN_ACT_SWIGLU 4

/* out[t][f] = act( sum_k x[t][k] w[f][k] + bias[f] ) + residual[t][f] */
typedef struct inkattn_linear_params {
    size_t struct_size;        /* = sizeof(inkattn_linear_params)                        */
    int32_t N_tok;             /* rows of x, >= 0                                        */
    int32_t K;                 /* input width: a multiple of 8, 8 .. 2^20                */
    int32_t F;                 /* output features, 1 .. 2^20                             */
    int32_t act;               /* INKATTN_ACT_*                                          */
    int32_t out_dtype;         /* INKATTN_DTYPE_BF16 (0) or INKATTN_DTYPE_F32 (1)        */
    const inkattn_bf16 *x;     /* [N_tok][K]; device memory of this GPU                  */
    const inkattn_bf16 *w;     /* [F][K] (SWIGLU: [2 F][K]); device memory of this GPU   */
    const float *bias;         /* nullable, [F] (SWIGLU: [2 F])                          */
    const inkattn_bf16 *residual;  /* nullable, [N_tok][F], added in fp32 before the     */
                                   /* rounding                                           */
    void *out;                 /* [N_tok][F], bf16 or fp32 per out_dtype                 */
    int32_t *dev_status;       /* nullable, see the conventions above                    */
} inkattn_linear_params;

/* Runs the linear layer.  x and w, which TMA may read, lie in device memory of the current
 * device, 16-byte aligned; residual and out must be 16-byte aligned.  out may be the residual
 * array itself (bf16), but overlaps no other input (INKATTN_ERR_INVALID_ARG). */
INKATTN_API inkattn_status inkattn_linear(const inkattn_linear_params *p, void *stream);

/* Products grouped by expert: the rows i in [expert_offsets[e], expert_offsets[e+1]) of out are
 *   out[i][f] = act( sum_k x[s][k] w[e][f][k] + bias[e][f] ),   s = row_token ? row_token[i] : i.
 * expert_offsets lies on the device, so the same call (or captured graph) serves any split of
 * the rows among the experts; an expert without rows costs nothing.  Rows at and behind
 * expert_offsets[E] are not written, and nothing depends on them.  An expert whose offsets are negative,
 * decrease, pass M or reach back behind an earlier expert's end is flagged
 * (INKATTN_ERR_DEVICE_BOUNDS) and its rows left as they were, and so is a row whose row_token
 * lies outside [0, N_x). */
#define INKATTN_MAX_EXPERTS 1024
typedef struct inkattn_grouped_linear_params {
    size_t struct_size;        /* = sizeof(inkattn_grouped_linear_params)                */
    int32_t E;                 /* experts, 1 .. INKATTN_MAX_EXPERTS                      */
    int32_t M;                 /* rows of out (capacity), >= 0                           */
    int32_t N_x;               /* rows of x; >= M where row_token is NULL                */
    int32_t K;                 /* input width: a multiple of 8, 8 .. 2^20                */
    int32_t F;                 /* output features, 1 .. 2^20                             */
    int32_t act;               /* INKATTN_ACT_*                                          */
    int32_t out_dtype;         /* INKATTN_DTYPE_BF16 (0) or INKATTN_DTYPE_F32 (1)        */
    const inkattn_bf16 *x;     /* [N_x][K]; device memory of this GPU                    */
    const inkattn_bf16 *w;     /* [E][F][K] (SWIGLU: [E][2 F][K]); device memory of this GPU */
    const float *bias;         /* nullable, [E][F] (SWIGLU: [E][2 F])                    */
    const int32_t *expert_offsets;  /* [E+1], non-decreasing, expert_offsets[E] <= M     */
    const int32_t *row_token;  /* nullable, [M]: the row of x that row i multiplies      */
    void *out;                 /* [M][F], bf16 or fp32 per out_dtype                     */
    int32_t *dev_status;       /* nullable                                               */
} inkattn_grouped_linear_params;

/* Runs the grouped products.  Rules of memory, alignment and overlap as inkattn_linear's. */
INKATTN_API inkattn_status inkattn_grouped_linear(const inkattn_grouped_linear_params *p, void *stream);

/* The router's choice.  Token t has E routed logits and, behind them, n_shared logits of
 * shared experts.  Its top_k routed experts are those of the largest logits, in descending
 * order, equal logits by the lower index first (a NaN counts as -infinity).  With
 *   s(l) = 1 / (1 + exp(-l))  (INKATTN_SCORE_SIGMOID)   or   exp(l)  (INKATTN_SCORE_SOFTMAX)
 * the weights of the chosen and the shared experts are scale * s(l) / (sum of their s(l)), in
 * fp32 (all zero where that sum is zero, as when every logit is -infinity), within
 * (16 + |l - m|) 2^-23 of the value, m the largest of their logits (sigmoid: or 0, if that is
 * less), and possibly 0 below 2^-125 |scale|.  The N_tok * top_k
 * (token, choice) pairs are then sorted by expert, stably in (token, choice) order:
 *   expert_offsets[e] = first row of expert e, row_token[i] = the token of row i (the row_token
 *   of inkattn_grouped_linear), token_rows[t][j] = the row of token t's j-th choice (the
 *   token_rows of inkattn_expert_combine). */
#define INKATTN_SCORE_SIGMOID 0
#define INKATTN_SCORE_SOFTMAX 1
#define INKATTN_MAX_TOP_K 16
#define INKATTN_MAX_SHARED 16
typedef struct inkattn_route_params {
    size_t struct_size;        /* = sizeof(inkattn_route_params)                         */
    int32_t N_tok;             /* tokens, >= 0 (0 writes expert_offsets alone); N_tok *  */
                               /* top_k <= 2^28                                          */
    int32_t E;                 /* routed experts, 1 .. INKATTN_MAX_EXPERTS               */
    int32_t n_shared;          /* shared experts, 0 .. INKATTN_MAX_SHARED                */
    int32_t top_k;             /* 1 .. min(E, INKATTN_MAX_TOP_K)                         */
    int32_t score;             /* INKATTN_SCORE_*                                        */
    float scale;               /* factor of the weights, finite                          */
    const float *logits;       /* [N_tok][E + n_shared]                                  */
    int32_t *topk_ids;         /* [N_tok][top_k]                                         */
    float *weights;            /* [N_tok][top_k + n_shared]                              */
    int32_t *expert_offsets;   /* [E+1]                                                  */
    int32_t *row_token;        /* [N_tok * top_k]                                        */
    int32_t *token_rows;       /* [N_tok][top_k]                                         */
} inkattn_route_params;

/* Bytes of workspace inkattn_route needs: 0 for small batches, or if the params are invalid. */
INKATTN_API size_t inkattn_route_workspace_bytes(const inkattn_route_params *p);

/* Runs the router.  All arrays 4-byte aligned, in memory of the current device; the outputs
 * overlap neither each other nor the logits.  workspace: device memory, 16-byte aligned, at
 * least inkattn_route_workspace_bytes bytes (nullable when that is 0), which overlap none of the
 * arrays; need not be cleared; calls whose GPU work overlaps need one each (two that share one
 * give wrong places, within the arrays all the same). */
INKATTN_API inkattn_status inkattn_route(const inkattn_route_params *p, void *workspace,
                                         size_t workspace_bytes, void *stream);

/* The weighted sum of each token's expert rows, in fp32, choices in order, then the shared
 * experts in order, rounded once to bf16:
 *   out[t] = sum_{j<top_k} weights[t][j] y[token_rows[t][j]] + sum_s weights[t][top_k+s] shared[s][t].
 * A choice whose token_rows entry is -1 (a dropped row) adds nothing; any other entry outside
 * [0, M) is flagged (INKATTN_ERR_DEVICE_BOUNDS) and adds nothing either. */
typedef struct inkattn_expert_combine_params {
    size_t struct_size;        /* = sizeof(inkattn_expert_combine_params)                */
    int32_t N_tok;             /* tokens, >= 0                                           */
    int32_t M;                 /* rows of y, >= 0                                        */
    int32_t F;                 /* width: a multiple of 8, 8 .. 2^20                      */
    int32_t top_k;             /* 1 .. INKATTN_MAX_TOP_K                                 */
    int32_t n_shared;          /* 0 .. INKATTN_MAX_SHARED                                */
    const inkattn_bf16 *y;     /* [M][F]                                                 */
    const inkattn_bf16 *shared;    /* [n_shared][N_tok][F] (nullable iff n_shared == 0)  */
    const float *weights;      /* [N_tok][top_k + n_shared]                              */
    const int32_t *token_rows; /* [N_tok][top_k]                                         */
    inkattn_bf16 *out;         /* [N_tok][F]                                             */
    int32_t *dev_status;       /* nullable                                               */
} inkattn_expert_combine_params;

/* Runs the sum.  y, shared and out must be 16-byte aligned; all arrays in memory of the current
 * device; out overlaps no input. */
INKATTN_API inkattn_status inkattn_expert_combine(const inkattn_expert_combine_params *p, void *stream);

/* ------------------------------------------------------------------------------
 * A verification step's end [VJ and VV: 8 chained MTP heads draft tokens, and the next step's decode
 * runs over a sequence's last token and its drafts].  Behind the decode: the probabilities of
 * the step's logits, the drafts that stand and the token behind them, and the conv states of
 * the rows kept.  The rejected rows of the KV cache need no undoing: they lie behind the
 * sequence's new length and are written again.
 * ------------------------------------------------------------------------------ */
#define INKATTN_MAX_VOCAB (1 << 20)

/* Probabilities of rows of logits, with t = temperature[row] (1 where temperature is NULL):
 *   probs[row][v] = exp((l_v - m) / t) / sum_w exp((l_w - m) / t),  m the row's largest logit;
 *   t = 0: 1 at the first of the largest logits, 0 elsewhere.
 * A NaN counts as -infinity; a row of -infinities gives zeros; of a row with infinite logits,
 * those alone share the 1.  A temperature that is negative, infinite or NaN is flagged
 * (INKATTN_ERR_DEVICE_BOUNDS) and its row written as zeros.  Relative error at most
 * (64 + V 2^-14 + 2 (m - l_v) / t) 2^-23 of a value, and possibly 0 below 2^-125 (finite logits
 * further apart than the largest float, and temperatures above 2^126 or below 2^-127, are less exact). */
typedef struct inkattn_token_probs_params {
    size_t struct_size;        /* = sizeof(inkattn_token_probs_params)                   */
    int32_t N_tok;             /* rows, 0 .. 2^24                                        */
    int32_t V;                 /* logits of a row, 1 .. INKATTN_MAX_VOCAB                */
    int32_t logits_dtype;      /* INKATTN_DTYPE_BF16 (0) or INKATTN_DTYPE_F32 (1)        */
    int64_t logits_stride;     /* elements from row to row, V .. 2^32                    */
    int64_t probs_stride;      /* elements from row to row, V .. 2^32                    */
    const void *logits;        /* [N_tok][logits_stride], bf16 or fp32                   */
    const float *temperature;  /* nullable, [N_tok]                                      */
    float *probs;              /* [N_tok][probs_stride]; what lies behind V is not written */
    int32_t *dev_status;       /* nullable                                               */
} inkattn_token_probs_params;

/* Runs the softmax.  Arrays aligned to their elements' size, in memory of the current device; probs
 * may be the logits array itself (fp32, the same stride), but overlaps no input otherwise (an array
 * is all from its first element to its last, what lies between its rows included). */
INKATTN_API inkattn_status inkattn_token_probs(const inkattn_token_probs_params *p, void *stream);

/* Verification of drafted tokens by rejection sampling.  Sequence b has the rows cu_seqlens_q[b]
 * .. cu_seqlens_q[b+1] - 1 of the step: its last token and its drafts, token_ids as the step took
 * them in.  Row i of a sequence holds the target's distribution p_i behind its token and, where
 * draft_p is given, the distribution q_i that the next row's draft x = token_ids[row + 1] was
 * drawn from (the last row's is not read).  Drafts are taken in order while
 *   u_accept[row] * q_i(x) < p_i(x)        (fp32; draft_p NULL: q_i(x) = 1, a draft without choice)
 * and the token behind them is drawn from max(p_i - q_i, 0) at the first row i whose draft does
 * not stand (draft_p NULL: from p_i without x), or from the last row's p_i where all do; where that
 * weight is zero everywhere, from p_i.  A probability outside [0, 1] counts as the nearer bound, a
 * NaN as 0, and the difference is one of fp32 numbers, rounded to nearest.
 *   Drawing: weights w_v are rounded to multiples of 2^-43 (ties to even) and summed as whole
 *   numbers, W in all; with U = floor(u_sample[b] 2^32) the token is the smallest v with w_0 + ..
 *   + w_v > floor(W U / 2^32).  The result depends on no order of sums, and is the same on
 *   every call and device.
 * n_new[b] = drafts that stand + 1: the step's new tokens, and the rows of the step that keep
 * their place (the n_keep of inkattn_conv_rollback); 0 for a sequence without rows.  out_tokens at
 * the sequence's rows: the drafts that stand, the drawn token, then -1.
 * Flagged (INKATTN_ERR_DEVICE_BOUNDS): a cu_seqlens_q out of range or decreasing (n_new 0, the
 * tokens not written), a draft outside [0, V) behind drafts that stand (does not stand, nothing is taken from p_i for it), a
 * row to draw from whose weights are all zero (token -1, n_new without it).  u values outside
 * [0, 1) count as the nearer bound (the largest float below 1), a NaN as 0. */
typedef struct inkattn_verify_drafts_params {
    size_t struct_size;        /* = sizeof(inkattn_verify_drafts_params)                 */
    int32_t B;                 /* sequences, 1 .. 2^20                                   */
    int32_t N_tok;             /* rows = cu_seqlens_q[B], 0 .. 2^24                      */
    int32_t V;                 /* vocabulary, 1 .. INKATTN_MAX_VOCAB                     */
    int64_t target_stride;     /* elements from row to row, V .. 2^32                    */
    int64_t draft_stride;      /* the same of draft_p (not read where that is NULL)      */
    const float *target_p;     /* [N_tok][target_stride]                                 */
    const float *draft_p;      /* nullable, [N_tok][draft_stride]                        */
    const int32_t *token_ids;  /* [N_tok]                                                */
    const int32_t *cu_seqlens_q;   /* [B+1]                                              */
    const float *u_accept;     /* [N_tok], in [0, 1)                                     */
    const float *u_sample;     /* [B], in [0, 1)                                         */
    int32_t *n_new;            /* [B]                                                    */
    int32_t *out_tokens;       /* [N_tok]                                                */
    int32_t *dev_status;       /* nullable                                               */
} inkattn_verify_drafts_params;

/* Runs the verification.  All arrays 4-byte aligned, in memory of the current device; the outputs
 * overlap neither each other nor an input (rows of a stride as for the softmax). */
INKATTN_API inkattn_status inkattn_verify_drafts(const inkattn_verify_drafts_params *p, void *stream);

/* The conv states behind the first n_keep[b] of a step's rows: with xs = the 3 rows of
 * state_before[slot], then the rows of x from cu_seqlens_q[b] on,
 *   state_after[slot][i] = xs[n_keep[b] + i],  i = 0 .. 2,  slot = state_slot[b],
 * for every conv of `states` (a layer's K, V, attention output and MLP output, say) in one
 * launch.  state_before is the state from before the step, which a call that updates its state
 * in place has overwritten: keep a copy, or let inkattn_qkvr_prologue write elsewhere.  Other slots
 * are not touched.  A cu_seqlens_q, slot or n_keep (0 .. the sequence's rows) out of range is
 * flagged (INKATTN_ERR_DEVICE_BOUNDS) and its sequence skipped. */
#define INKATTN_ROLLBACK_MAX_STATES 8
typedef struct inkattn_conv_rows {
    int32_t C;                 /* channels: a multiple of 8, 8 .. 2^20                   */
    int64_t x_stride;          /* elements from row to row of x, C .. 2^32, a multiple of 8 */
    const inkattn_bf16 *x;     /* [N_tok][x_stride], the conv's input rows of the step   */
    const inkattn_bf16 *state_before;  /* [num_state_slots][3][C]                        */
    inkattn_bf16 *state_after;         /* [num_state_slots][3][C]; may be state_before   */
} inkattn_conv_rows;
typedef struct inkattn_conv_rollback_params {
    size_t struct_size;        /* = sizeof(inkattn_conv_rollback_params)                 */
    int32_t B;                 /* sequences, 1 .. 65535                                  */
    int32_t N_tok;             /* rows = cu_seqlens_q[B], >= 0                           */
    int32_t num_state_slots;   /* capacity in slots (bounds check), >= 1                 */
    int32_t n_states;          /* 1 .. INKATTN_ROLLBACK_MAX_STATES                       */
    const int32_t *cu_seqlens_q;   /* [B+1]                                              */
    const int32_t *state_slot;     /* [B], distinct values in [0, num_state_slots)       */
    const int32_t *n_keep;         /* [B]                                                */
    int32_t *dev_status;           /* nullable                                           */
    inkattn_conv_rows states[INKATTN_ROLLBACK_MAX_STATES];
} inkattn_conv_rollback_params;

/* Runs the rollback.  x (nullable where N_tok is 0) and the states 16-byte aligned, all arrays in
 * memory of the current device; a state_after overlaps no other array, its own state_before either
 * exactly or not at all. */
INKATTN_API inkattn_status inkattn_conv_rollback(const inkattn_conv_rollback_params *p, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* INKATTN_H */
