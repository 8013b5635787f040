// api.cu -- the extern "C" entry points of libinkattn.so: host-side validation, TMA
// descriptor setup, the decode split heuristic, and the launches.
//
// Nothing here computes on the host: every step of the path runs in the kernels of
// prologue.cu, qkvr.cu, output_conv.cu, prefill_tc.cu, decode.cu, linear.cu, route.cu, verify.cu and rollback.cu.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <mutex>

#include "../../include/inkattn.h"
#include "internal.h"

namespace inkattn {
namespace {

constexpr int kMaxDevices = 64;
constexpr uint64_t kWaitLimitNsDefault = 1000000000ull;   // 1 s, as the kernels' default

// ---------------------------------------------------------------- device checks

std::atomic<int> g_dev_ok[kMaxDevices];       // 0 unknown, 1 sm_103, 2 other
std::atomic<int> g_dev_sms[kMaxDevices];

inkattn_status check_device(int *sms_out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return INKATTN_ERR_CUDA;
    if (dev < 0 || dev >= kMaxDevices) return INKATTN_ERR_UNSUPPORTED;
    int ok = g_dev_ok[dev].load(std::memory_order_acquire);
    if (ok == 0) {
        int major = 0, minor = 0, sms = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return INKATTN_ERR_CUDA;
        g_dev_sms[dev].store(sms, std::memory_order_relaxed);
        ok = (major == 10 && minor == 3) ? 1 : 2;
        g_dev_ok[dev].store(ok, std::memory_order_release);
    }
    if (sms_out) *sms_out = g_dev_sms[dev].load(std::memory_order_relaxed);
    return ok == 1 ? INKATTN_OK : INKATTN_ERR_UNSUPPORTED;
}

// ---------------------------------------------------------------- TMA encode

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    std::call_once(g_encode_once, [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
                cudaSuccess && q == cudaDriverEntryPointSuccess)
            g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    return g_encode;
}

bool aligned(const void *ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) == 0; }

// ---------------------------------------------------------------- validation

// The cache's element type, and the scales that a cache of codes has.
bool valid_kv(int32_t kv_dtype, const void *k_scale, const void *v_scale) {
    if (kv_dtype == INKATTN_KV_BF16) return true;
    return (kv_dtype == INKATTN_KV_E4M3 || kv_dtype == INKATTN_KV_I4) && k_scale && v_scale && aligned(k_scale, 16) &&
           aligned(v_scale, 16);
}
// Bytes of a cache row of one head.
size_t kv_row_bytes(int32_t kv_dtype) {
    return kv_dtype == INKATTN_KV_I4 ? kHeadDim / 2 : kv_dtype == INKATTN_KV_E4M3 ? kHeadDim : kHeadDim * 2;
}

inkattn_status validate_prologue(const inkattn_prologue_params *p) {
    if (!p || p->struct_size != sizeof(inkattn_prologue_params)) return INKATTN_ERR_INVALID_ARG;
    if (p->B < 1 || p->N_tok < 0 || p->max_seqlen_q < 0 || p->Hq < 1 || p->Hkv < 1 ||
        p->Hq % p->Hkv != 0 || p->num_blocks < 1 || p->num_state_slots < 1 || !(p->eps >= 0.f))
        return INKATTN_ERR_INVALID_ARG;
    if (p->N_tok > 0 && p->max_seqlen_q < 1) return INKATTN_ERR_INVALID_ARG;
    if (p->B > 65535 || p->Hq > 65535) return INKATTN_ERR_INVALID_ARG;   // (query rows of a tile: 32-bit offsets)
    if ((long long)p->num_blocks * 64 > INT_MAX) return INKATTN_ERR_INVALID_ARG;
    if (p->head_dim != kHeadDim || p->block_size != kBlock) return INKATTN_ERR_UNSUPPORTED;
    const void *ptrs16[] = {p->q, p->k, p->v, p->conv_state_k, p->conv_state_v, p->q_out,
                            p->k_cache, p->v_cache};
    for (const void *ptr : ptrs16)
        if (!ptr || !aligned(ptr, 16)) return INKATTN_ERR_INVALID_ARG;
    const void *ptrs4[] = {p->conv_w_k, p->conv_w_v, p->q_norm_w, p->k_norm_w, p->cu_seqlens_q,
                           p->state_slot, p->slot_mapping};
    for (const void *ptr : ptrs4)
        if (!ptr || !aligned(ptr, 4)) return INKATTN_ERR_INVALID_ARG;
    if (p->dev_status && !aligned(p->dev_status, 4)) return INKATTN_ERR_INVALID_ARG;
    if (!valid_kv(p->kv_dtype, p->k_scale, p->v_scale)) return INKATTN_ERR_INVALID_ARG;
    return INKATTN_OK;
}

inkattn_status validate_output_conv(const inkattn_output_conv_params *p) {
    if (!p || p->struct_size != sizeof(inkattn_output_conv_params)) return INKATTN_ERR_INVALID_ARG;
    if (p->B < 1 || p->B > 65535 || p->N_tok < 0 || p->max_seqlen_q < 0 || p->num_state_slots < 1 ||
        !(p->eps >= 0.f))
        return INKATTN_ERR_INVALID_ARG;
    if (p->D < 8 || p->D > 32768 || p->D % 8 != 0) return INKATTN_ERR_INVALID_ARG;
    if (p->N_tok > 0 && p->max_seqlen_q < 1) return INKATTN_ERR_INVALID_ARG;
    const void *ptrs16[] = {p->y, p->conv_w, p->norm_w, p->conv_state, p->residual, p->h_out, p->out};
    for (const void *ptr : ptrs16)
        if (!ptr || !aligned(ptr, 16)) return INKATTN_ERR_INVALID_ARG;
    const void *ptrs4[] = {p->cu_seqlens_q, p->state_slot};
    for (const void *ptr : ptrs4)
        if (!ptr || !aligned(ptr, 4)) return INKATTN_ERR_INVALID_ARG;
    if (p->dev_status && !aligned(p->dev_status, 4)) return INKATTN_ERR_INVALID_ARG;
    // h_out may be the residual array itself, but no other output may overlap an input
    const size_t row = (size_t)p->N_tok * p->D * 2;
    auto overlap = [](const void *a, size_t na, const void *b, size_t nb) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
        return na && nb && x < y + nb && y < x + na;
    };
    if (overlap(p->out, row, p->y, row) || overlap(p->out, row, p->residual, row) ||
        overlap(p->out, row, p->h_out, row) || overlap(p->h_out, row, p->y, row) ||
        (p->h_out != p->residual && overlap(p->h_out, row, p->residual, row)))
        return INKATTN_ERR_INVALID_ARG;
    return INKATTN_OK;
}

inkattn_status validate_qkvr(const inkattn_qkvr_params *p) {
    if (!p || p->struct_size != sizeof(inkattn_qkvr_params)) return INKATTN_ERR_INVALID_ARG;
    if (p->B < 1 || p->B > INKATTN_QKVR_MAX_SEQS || p->N_tok < 0 || p->max_seqlen_q < 0 || p->Hq < 1 ||
        p->Hkv < 1 || p->Hq % p->Hkv != 0 || p->Hq > 1024 || p->num_blocks < 1 || p->num_state_slots < 1 ||
        !(p->eps >= 0.f))
        return INKATTN_ERR_INVALID_ARG;
    if (p->N_tok > 0 && p->max_seqlen_q < 1) return INKATTN_ERR_INVALID_ARG;
    if (p->d_r < 1 || p->d_r > 1024 || ((long long)p->Hq * p->d_r) % 8 != 0) return INKATTN_ERR_INVALID_ARG;
    if (p->d_model < 8 || p->d_model % 8 != 0 || p->d_model > (1 << 20)) return INKATTN_ERR_INVALID_ARG;
    if ((long long)p->num_blocks * 64 > INT_MAX) return INKATTN_ERR_INVALID_ARG;
    if (p->head_dim != kHeadDim || p->block_size != kBlock) return INKATTN_ERR_UNSUPPORTED;
    const void *ptrs16[] = {p->x, p->w, p->conv_state_k_in, p->conv_state_v_in, p->conv_state_k_out,
                            p->conv_state_v_out, p->q_out, p->r_out, p->k_cache, p->v_cache};
    for (const void *ptr : ptrs16)
        if (!ptr || !aligned(ptr, 16)) return INKATTN_ERR_INVALID_ARG;
    const void *ptrs4[] = {p->conv_w_k, p->conv_w_v, p->q_norm_w, p->k_norm_w, p->cu_seqlens_q,
                           p->state_slot, p->slot_mapping};
    for (const void *ptr : ptrs4)
        if (!ptr || !aligned(ptr, 4)) return INKATTN_ERR_INVALID_ARG;
    if (p->dev_status && !aligned(p->dev_status, 4)) return INKATTN_ERR_INVALID_ARG;
    if (p->y_out && !aligned(p->y_out, 16)) return INKATTN_ERR_INVALID_ARG;
    if (!valid_kv(p->kv_dtype, p->k_scale, p->v_scale)) return INKATTN_ERR_INVALID_ARG;
    // the new state is written while a sequence's first tile still reads the old one,
    // unless every sequence fits one tile
    if ((p->conv_state_k_out == p->conv_state_k_in || p->conv_state_v_out == p->conv_state_v_in) &&
        p->max_seqlen_q > INKATTN_QKVR_TILE_TOKENS)
        return INKATTN_ERR_INVALID_ARG;
    // no output overlaps an input or another output (in == out for the states excepted)
    const size_t F = (size_t)(p->Hq + 2 * p->Hkv) * kHeadDim + (size_t)p->Hq * p->d_r;
    const size_t st = (size_t)p->num_state_slots * 3 * p->Hkv * kHeadDim * 2;
    const size_t cache = (size_t)p->num_blocks * p->Hkv * 64 * kv_row_bytes(p->kv_dtype);
    struct Range { const void *a; size_t n; };
    const Range ins[] = {{p->x, (size_t)p->N_tok * p->d_model * 2}, {p->w, F * p->d_model * 2},
                         {p->conv_state_k_in, st}, {p->conv_state_v_in, st}};
    const Range outs[] = {{p->q_out, (size_t)p->N_tok * p->Hq * kHeadDim * 2},
                          {p->r_out, (size_t)p->N_tok * p->Hq * p->d_r * 2},
                          {p->k_cache, cache}, {p->v_cache, cache},
                          {p->conv_state_k_out, st}, {p->conv_state_v_out, st},
                          {p->y_out, p->y_out ? (size_t)p->N_tok * F * 2 : 0}};
    auto overlap = [](const Range &x, const Range &y) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(x.a), b = reinterpret_cast<uintptr_t>(y.a);
        return x.n && y.n && a < b + y.n && b < a + x.n;
    };
    constexpr int kOuts = sizeof(outs) / sizeof(outs[0]);
    for (int o = 0; o < kOuts; ++o) {
        for (int i = 0; i < 4; ++i) {
            const bool same_state = (o == 4 && i == 2 && outs[o].a == ins[i].a) ||
                                    (o == 5 && i == 3 && outs[o].a == ins[i].a);
            if (!same_state && overlap(outs[o], ins[i])) return INKATTN_ERR_INVALID_ARG;
        }
        for (int o2 = o + 1; o2 < kOuts; ++o2)
            if (overlap(outs[o], outs[o2])) return INKATTN_ERR_INVALID_ARG;
    }
    return INKATTN_OK;
}

// x and w are read by TMA: device memory of the current device (as for validate_locations)
inkattn_status validate_qkvr_locations(const inkattn_qkvr_params *p) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return INKATTN_ERR_INVALID_ARG;
    }
    const void *ptrs[] = {p->x, p->w};
    for (const void *ptr : ptrs) {
        cudaPointerAttributes a;
        if (cudaPointerGetAttributes(&a, ptr) != cudaSuccess) {
            (void)cudaGetLastError();
            return INKATTN_ERR_INVALID_ARG;
        }
        if (a.type != cudaMemoryTypeDevice || a.device != dev) return INKATTN_ERR_INVALID_ARG;
    }
    return INKATTN_OK;
}

inkattn_status validate_attn(const inkattn_attn_params *p) {
    if (!p || p->struct_size != sizeof(inkattn_attn_params)) return INKATTN_ERR_INVALID_ARG;
    if (p->B < 1 || p->B > 65535 || p->N_tok < 0 || p->max_seqlen_q < 0 || p->max_seqlen_k < 0 ||
        p->Hq < 1 || p->Hkv < 1 || p->Hq % p->Hkv != 0 || p->Hq > 65535 || p->num_blocks < 1 ||
        p->max_blocks_per_seq < 1 || p->rel_extent < 0 || p->window < 0)
        return INKATTN_ERR_INVALID_ARG;
    if (p->N_tok > 0 && (p->max_seqlen_q < 1 || p->max_seqlen_k < p->max_seqlen_q))
        return INKATTN_ERR_INVALID_ARG;
    if ((long long)p->max_blocks_per_seq * kBlock < p->max_seqlen_k) return INKATTN_ERR_INVALID_ARG;
    if ((long long)p->num_blocks * p->Hkv * kBlock >= (1ll << 31)) return INKATTN_ERR_INVALID_ARG;
    if (p->head_dim != kHeadDim || p->block_size != kBlock) return INKATTN_ERR_UNSUPPORTED;
    if (p->out_dtype != INKATTN_DTYPE_BF16 && p->out_dtype != INKATTN_DTYPE_F32) return INKATTN_ERR_INVALID_ARG;
    if (!(p->softmax_scale == p->softmax_scale) || !(p->log_scale_base == p->log_scale_base))
        return INKATTN_ERR_INVALID_ARG;
    const void *ptrs16[] = {p->q, p->k_cache, p->v_cache, p->out};
    for (const void *ptr : ptrs16)
        if (!ptr || !aligned(ptr, 16)) return INKATTN_ERR_INVALID_ARG;
    const void *ptrs4[] = {p->cu_seqlens_q, p->seqlen_k, p->block_table};
    for (const void *ptr : ptrs4)
        if (!ptr || !aligned(ptr, 4)) return INKATTN_ERR_INVALID_ARG;
    if (p->lse && !aligned(p->lse, 4)) return INKATTN_ERR_INVALID_ARG;
    if (p->dev_status && !aligned(p->dev_status, 4)) return INKATTN_ERR_INVALID_ARG;
    if (!valid_kv(p->kv_dtype, p->k_scale, p->v_scale)) return INKATTN_ERR_INVALID_ARG;
    if (p->rel_extent > 0) {
        if (p->d_r != 32) return INKATTN_ERR_UNSUPPORTED;
        if (!p->r || !p->P || !aligned(p->r, 16) || !aligned(p->P, 16)) return INKATTN_ERR_INVALID_ARG;
    }
    return INKATTN_OK;
}

// q, k_cache and v_cache are read by TMA through tensor maps, and the prefill kernel
// multicasts each K/V tile to the two CTAs of a head pair: the maps must cover memory of
// this GPU alone.  Each must be device memory of the current device; host memory (pinned
// or not), managed memory and another GPU's memory reached through unified addressing are
// rejected.  A pointer whose location the runtime cannot report is rejected too.
inkattn_status validate_locations(const inkattn_attn_params *p) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return INKATTN_ERR_INVALID_ARG;
    }
    const bool codes = p->kv_dtype != INKATTN_KV_BF16;
    const void *q = p->q;
    const void *ptrs[] = {q, p->k_cache, p->v_cache, codes ? static_cast<const void *>(p->k_scale) : q,
                          codes ? static_cast<const void *>(p->v_scale) : q};
    for (const void *ptr : ptrs) {
        cudaPointerAttributes a;
        if (cudaPointerGetAttributes(&a, ptr) != cudaSuccess) {
            (void)cudaGetLastError();
            return INKATTN_ERR_INVALID_ARG;
        }
        if (a.type != cudaMemoryTypeDevice || a.device != dev) return INKATTN_ERR_INVALID_ARG;
    }
    return INKATTN_OK;
}

// Device memory of the current device: what TMA reads; where nothing is read by TMA, one or two arrays of a
// call, so that a call made under another current device is refused; every array (dev_status aside) of a
// verification step's end.
//
// Arrays of one allocation are told by its range, so that a call of many arrays asks about few: a rollback of
// eight convs takes 3.5 us of the host's time, 5.7 with its 27 arrays asked about one by one.
PFN_cuPointerGetAttributes_v7000 pointer_attributes() {
    static const PFN_cuPointerGetAttributes_v7000 f = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool found = cudaGetDriverEntryPointByVersion("cuPointerGetAttributes", &fn, 7000, cudaEnableDefault, &q) ==
                               cudaSuccess && q == cudaDriverEntryPointSuccess;
        return found ? reinterpret_cast<PFN_cuPointerGetAttributes_v7000>(fn) : nullptr;
    }();
    return f;
}
inkattn_status validate_on_device(const void *const *ptrs, int n) {
    int dev = -1;
    const PFN_cuPointerGetAttributes_v7000 query = pointer_attributes();
    if (!query || cudaGetDevice(&dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return INKATTN_ERR_INVALID_ARG;
    }
    constexpr int kKnown = 4;                          // allocations of this device seen in this call
    CUdeviceptr known[kKnown] = {};
    size_t known_bytes[kKnown] = {};
    int next = 0;
    for (int i = 0; i < n; ++i) {
        const CUdeviceptr ptr = reinterpret_cast<CUdeviceptr>(ptrs[i]);
        bool seen = false;
        for (int k = 0; k < kKnown; ++k) seen = seen || ptr - known[k] < known_bytes[k];
        if (seen) continue;
        unsigned int type = 0, managed = 0;
        int where = -1;
        CUdeviceptr start = 0;
        size_t bytes = 0;
        CUpointer_attribute names[] = {CU_POINTER_ATTRIBUTE_MEMORY_TYPE, CU_POINTER_ATTRIBUTE_IS_MANAGED,
                                       CU_POINTER_ATTRIBUTE_DEVICE_ORDINAL, CU_POINTER_ATTRIBUTE_RANGE_START_ADDR,
                                       CU_POINTER_ATTRIBUTE_RANGE_SIZE};
        void *values[] = {&type, &managed, &where, &start, &bytes};
        if (query(5, names, values, ptr) != CUDA_SUCCESS) return INKATTN_ERR_INVALID_ARG;
        if (type != CU_MEMORYTYPE_DEVICE || managed || where != dev) return INKATTN_ERR_INVALID_ARG;
        known[next] = start;                           // (0 bytes where the driver does not say)
        known_bytes[next] = bytes;
        next = (next + 1) % kKnown;
    }
    return INKATTN_OK;
}

struct Range {
    const void *a;
    size_t n;
};
bool overlap(const Range &x, const Range &y) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x.a), b = reinterpret_cast<uintptr_t>(y.a);
    // (by distances: rows of a wide stride may claim more than lies behind their address)
    return x.a && y.a && x.n && y.n && (a <= b ? b - a < x.n : a - b < y.n);
}

// Sizes, types and alignment that the linear layer and the grouped products share.  Arrays of
// no rows may be NULL.
inkattn_status validate_product(int rows, int K, int F, int act, int out_dtype, const void *x, const void *w, const void *bias,
                                const void *residual, const void *out, const void *dev_status) {
    if (K < 8 || K % 8 != 0 || K > (1 << 20) || F < 1 || F > (1 << 20)) return INKATTN_ERR_INVALID_ARG;
    if (act < INKATTN_ACT_NONE || act > INKATTN_ACT_SWIGLU) return INKATTN_ERR_INVALID_ARG;
    if (out_dtype != INKATTN_DTYPE_BF16 && out_dtype != INKATTN_DTYPE_F32) return INKATTN_ERR_INVALID_ARG;
    if (!w || (rows > 0 && (!x || !out)) || !aligned(x, 16) || !aligned(w, 16) || !aligned(out, 16))
        return INKATTN_ERR_INVALID_ARG;
    if ((bias && !aligned(bias, 4)) || (residual && !aligned(residual, 16)) || (dev_status && !aligned(dev_status, 4)))
        return INKATTN_ERR_INVALID_ARG;
    return INKATTN_OK;
}

inkattn_status validate_linear(const inkattn_linear_params *p) {
    if (!p || p->struct_size != sizeof(inkattn_linear_params) || p->N_tok < 0) return INKATTN_ERR_INVALID_ARG;
    const inkattn_status st = validate_product(p->N_tok, p->K, p->F, p->act, p->out_dtype, p->x, p->w, p->bias,
                                               p->residual, p->out, p->dev_status);
    if (st != INKATTN_OK) return st;
    const size_t elems = (size_t)p->N_tok * p->F, size = p->out_dtype == INKATTN_DTYPE_F32 ? 4 : 2;
    const size_t wrows = (size_t)p->F * (p->act == INKATTN_ACT_SWIGLU ? 2 : 1);
    const Range out = {p->out, elems * size};
    const Range ins[] = {{p->x, (size_t)p->N_tok * p->K * 2}, {p->w, wrows * p->K * 2}, {p->bias, wrows * 4},
                         {p->dev_status, 4}};
    for (const Range &in : ins)
        if (overlap(out, in)) return INKATTN_ERR_INVALID_ARG;
    const bool in_place = p->residual == p->out && p->out_dtype == INKATTN_DTYPE_BF16;
    if (!in_place && overlap(out, {p->residual, elems * 2})) return INKATTN_ERR_INVALID_ARG;
    return INKATTN_OK;
}

inkattn_status validate_grouped_linear(const inkattn_grouped_linear_params *p) {
    if (!p || p->struct_size != sizeof(inkattn_grouped_linear_params) || p->E < 1 || p->E > INKATTN_MAX_EXPERTS ||
        p->M < 0 || p->N_x < 0)
        return INKATTN_ERR_INVALID_ARG;
    const inkattn_status st = validate_product(p->M, p->K, p->F, p->act, p->out_dtype, p->x, p->w, p->bias, nullptr,
                                               p->out, p->dev_status);
    if (st != INKATTN_OK) return st;
    if (p->M > 0 && (p->row_token ? p->N_x < 1 : p->N_x < p->M)) return INKATTN_ERR_INVALID_ARG;
    if (!p->expert_offsets || !aligned(p->expert_offsets, 4) || (p->row_token && !aligned(p->row_token, 4)))
        return INKATTN_ERR_INVALID_ARG;
    const size_t size = p->out_dtype == INKATTN_DTYPE_F32 ? 4 : 2;
    const size_t wrows = (size_t)p->E * p->F * (p->act == INKATTN_ACT_SWIGLU ? 2 : 1);
    const Range out = {p->out, (size_t)p->M * p->F * size};
    const Range ins[] = {{p->x, (size_t)p->N_x * p->K * 2}, {p->w, wrows * p->K * 2}, {p->bias, wrows * 4},
                         {p->expert_offsets, (size_t)(p->E + 1) * 4}, {p->row_token, (size_t)p->M * 4},
                         {p->dev_status, 4}};
    for (const Range &in : ins)
        if (overlap(out, in)) return INKATTN_ERR_INVALID_ARG;
    return INKATTN_OK;
}

inkattn_status validate_route(const inkattn_route_params *p, const void *workspace, size_t workspace_bytes) {
    if (!p || p->struct_size != sizeof(inkattn_route_params) || p->N_tok < 0 || p->E < 1 ||
        p->E > INKATTN_MAX_EXPERTS || p->n_shared < 0 || p->n_shared > INKATTN_MAX_SHARED || p->top_k < 1 ||
        p->top_k > INKATTN_MAX_TOP_K || p->top_k > p->E || !std::isfinite(p->scale))
        return INKATTN_ERR_INVALID_ARG;
    if (p->score != INKATTN_SCORE_SIGMOID && p->score != INKATTN_SCORE_SOFTMAX) return INKATTN_ERR_INVALID_ARG;
    if ((long long)p->N_tok * p->top_k > (1ll << 28)) return INKATTN_ERR_INVALID_ARG;
    if (!p->expert_offsets || !aligned(p->expert_offsets, 4)) return INKATTN_ERR_INVALID_ARG;
    const void *ptrs[] = {p->logits, p->topk_ids, p->weights, p->row_token, p->token_rows};
    for (const void *ptr : ptrs)
        if ((p->N_tok > 0 && !ptr) || !aligned(ptr, 4)) return INKATTN_ERR_INVALID_ARG;
    const size_t T = (size_t)p->N_tok;
    const Range r[] = {{p->logits, T * (p->E + p->n_shared) * 4}, {p->topk_ids, T * p->top_k * 4},
                       {p->weights, T * (p->top_k + p->n_shared) * 4}, {p->expert_offsets, (size_t)(p->E + 1) * 4},
                       {p->row_token, T * p->top_k * 4}, {p->token_rows, T * p->top_k * 4}, {workspace, workspace_bytes}};
    for (int i = 0; i < 7; ++i)
        for (int j = i + 1; j < 7; ++j)
            if (overlap(r[i], r[j])) return INKATTN_ERR_INVALID_ARG;
    return INKATTN_OK;
}

inkattn_status validate_expert_combine(const inkattn_expert_combine_params *p) {
    if (!p || p->struct_size != sizeof(inkattn_expert_combine_params) || p->N_tok < 0 || p->M < 0 || p->F < 8 ||
        p->F % 8 != 0 || p->F > (1 << 20) || p->top_k < 1 || p->top_k > INKATTN_MAX_TOP_K || p->n_shared < 0 ||
        p->n_shared > INKATTN_MAX_SHARED)
        return INKATTN_ERR_INVALID_ARG;
    if ((long long)p->N_tok * ((p->F + 1023) / 1024) > INT_MAX) return INKATTN_ERR_INVALID_ARG;   // (the grid)
    const bool some = p->N_tok > 0;
    if ((p->M > 0 && !p->y) || (some && !p->out) || (some && p->n_shared > 0 && !p->shared) || !aligned(p->y, 16) ||
        !aligned(p->out, 16) || !aligned(p->shared, 16))
        return INKATTN_ERR_INVALID_ARG;
    const void *ptrs4[] = {p->weights, p->token_rows};
    for (const void *ptr : ptrs4)
        if ((some && !ptr) || !aligned(ptr, 4)) return INKATTN_ERR_INVALID_ARG;
    if (p->dev_status && !aligned(p->dev_status, 4)) return INKATTN_ERR_INVALID_ARG;
    const size_t T = (size_t)p->N_tok, F = (size_t)p->F;
    const Range out = {p->out, T * F * 2};
    const Range ins[] = {{p->y, (size_t)p->M * F * 2}, {p->shared, p->n_shared * T * F * 2},
                         {p->weights, T * (p->top_k + p->n_shared) * 4}, {p->token_rows, T * p->top_k * 4},
                         {p->dev_status, 4}};
    for (const Range &in : ins)
        if (overlap(out, in)) return INKATTN_ERR_INVALID_ARG;
    return INKATTN_OK;
}

// Bytes that `rows` rows of `width` elements of `size` bytes span, `stride` elements apart.
size_t span(int64_t rows, int64_t stride, int64_t width, size_t size) {
    return rows > 0 ? ((size_t)(rows - 1) * stride + width) * size : 0;
}
constexpr int64_t kMaxRowStride = 1ll << 32;       // (spans stay below 2^64)

inkattn_status validate_token_probs(const inkattn_token_probs_params *p) {
    if (!p || p->struct_size != sizeof(inkattn_token_probs_params) || p->N_tok < 0 || p->N_tok > (1 << 24) || p->V < 1 ||
        p->V > INKATTN_MAX_VOCAB || p->logits_stride < p->V || p->probs_stride < p->V ||
        p->logits_stride > kMaxRowStride || p->probs_stride > kMaxRowStride)
        return INKATTN_ERR_INVALID_ARG;
    if (p->logits_dtype != INKATTN_DTYPE_BF16 && p->logits_dtype != INKATTN_DTYPE_F32) return INKATTN_ERR_INVALID_ARG;
    const size_t size = p->logits_dtype == INKATTN_DTYPE_F32 ? 4 : 2;
    if ((p->N_tok > 0 && (!p->logits || !p->probs)) || !aligned(p->logits, size) || !aligned(p->probs, 4) ||
        !aligned(p->temperature, 4) || !aligned(p->dev_status, 4))
        return INKATTN_ERR_INVALID_ARG;
    const Range out = {p->probs, span(p->N_tok, p->probs_stride, p->V, 4)};
    const bool in_place = p->logits == p->probs && size == 4 && p->logits_stride == p->probs_stride;
    const Range ins[] = {{in_place ? nullptr : p->logits, span(p->N_tok, p->logits_stride, p->V, size)},
                         {p->temperature, (size_t)p->N_tok * 4}, {p->dev_status, 4}};
    for (const Range &in : ins)
        if (overlap(out, in)) return INKATTN_ERR_INVALID_ARG;
    return INKATTN_OK;
}

inkattn_status validate_verify_drafts(const inkattn_verify_drafts_params *p) {
    if (!p || p->struct_size != sizeof(inkattn_verify_drafts_params) || p->B < 1 || p->B > (1 << 20) || p->N_tok < 0 ||
        p->N_tok > (1 << 24) || p->V < 1 || p->V > INKATTN_MAX_VOCAB || p->target_stride < p->V ||
        p->target_stride > kMaxRowStride)
        return INKATTN_ERR_INVALID_ARG;
    if (p->draft_p && (p->draft_stride < p->V || p->draft_stride > kMaxRowStride)) return INKATTN_ERR_INVALID_ARG;
    const bool some = p->N_tok > 0;
    if (!p->cu_seqlens_q || !p->n_new || !p->u_sample ||
        (some && (!p->target_p || !p->token_ids || !p->u_accept || !p->out_tokens)))
        return INKATTN_ERR_INVALID_ARG;
    const size_t T = (size_t)p->N_tok, B = (size_t)p->B;
    const Range r[] = {{p->n_new, B * 4}, {p->out_tokens, T * 4}, {p->dev_status, 4}, {p->cu_seqlens_q, (B + 1) * 4},
                       {p->token_ids, T * 4}, {p->u_accept, T * 4}, {p->u_sample, B * 4},
                       {p->target_p, span(p->N_tok, p->target_stride, p->V, 4)},
                       {p->draft_p, p->draft_p ? span(p->N_tok, p->draft_stride, p->V, 4) : 0}};
    for (const Range &x : r)
        if (!aligned(x.a, 4)) return INKATTN_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i)                    // what is written
        for (int j = i + 1; j < 9; ++j)
            if (overlap(r[i], r[j])) return INKATTN_ERR_INVALID_ARG;
    return INKATTN_OK;
}

inkattn_status validate_conv_rollback(const inkattn_conv_rollback_params *p) {
    if (!p || p->struct_size != sizeof(inkattn_conv_rollback_params) || p->B < 1 || p->B > 65535 || p->N_tok < 0 ||
        p->num_state_slots < 1 || p->n_states < 1 || p->n_states > INKATTN_ROLLBACK_MAX_STATES)
        return INKATTN_ERR_INVALID_ARG;
    constexpr int kOthers = 4;
    Range r[kOthers + 3 * INKATTN_ROLLBACK_MAX_STATES] = {{p->cu_seqlens_q, ((size_t)p->B + 1) * 4},
                                                          {p->state_slot, (size_t)p->B * 4},
                                                          {p->n_keep, (size_t)p->B * 4}, {p->dev_status, 4}};
    for (int i = 0; i < kOthers; ++i)
        if ((i < 3 && !r[i].a) || !aligned(r[i].a, 4)) return INKATTN_ERR_INVALID_ARG;
    int n = kOthers;
    for (int s = 0; s < p->n_states; ++s) {
        const inkattn_conv_rows &c = p->states[s];
        if (c.C < 8 || c.C % 8 != 0 || c.C > (1 << 20) || c.x_stride < c.C || c.x_stride % 8 != 0 ||
            c.x_stride > kMaxRowStride)
            return INKATTN_ERR_INVALID_ARG;
        if ((p->N_tok > 0 && !c.x) || !c.state_before || !c.state_after || !aligned(c.x, 16) ||
            !aligned(c.state_before, 16) || !aligned(c.state_after, 16))
            return INKATTN_ERR_INVALID_ARG;
        const size_t bytes = (size_t)p->num_state_slots * 3 * c.C * 2;
        r[n++] = {c.x, span(p->N_tok, c.x_stride, c.C, 2)};
        r[n++] = {c.state_before, bytes};
        r[n++] = {c.state_after, bytes};
    }
    for (int o = kOthers + 2; o < n; o += 3)       // every state_after against everything else
        for (int i = 0; i < n; ++i) {
            const bool in_place = i == o - 1 && r[i].a == r[o].a;
            if (i != o && !in_place && overlap(r[o], r[i])) return INKATTN_ERR_INVALID_ARG;
        }
    return INKATTN_OK;
}

AttnScalars scalars(const inkattn_attn_params &p) {
    AttnScalars s;
    s.scale = p.softmax_scale > 0.f ? p.softmax_scale : 1.0f / sqrtf((float)kHeadDim);
    s.group = p.Hq / p.Hkv;
    return s;
}

inkattn_status launch_status(cudaError_t e) { return e == cudaSuccess ? INKATTN_OK : INKATTN_ERR_CUDA; }

}  // namespace

namespace {

// Decode split heuristic over a 4-bit cache, where a CTA's own steps set its pace and not HBM.  S parts of equal
// cost, one CTA an SM; or two parts cut at the band (csrc/decode_tc.cu), whose CTAs run beside each other.
// In microseconds: a CTA starts and drains in 9, takes 0.5 for a block and kI4BandCost times that for one of the
// band; the combine of S parts takes 2 + 0.27 S and its bytes at HBM's rate.  Fitted to a slower kernel: the
// present one starts and drains in 5, takes 0.5 for a block and 4.5 times that in the band, so that times come
// out too long, but the choice mostly stands.  GB300, 1 to 32 parts: in nine batches of one to 64 sequences with
// 1000 to 32768 keys it is the best or within 2% of it; in sixteen drawn ones within 11%, but for two of
// lengths far apart (28 us for 24, 89 for 39): every sequence is taken to be as long as the longest.
int pick_splits_i4(const inkattn_attn_params &p, int num_sms) {
    constexpr double kStart = 9.0, kBlockUs = 0.5;
    long long nblk = ((long long)p.max_seqlen_k + kBlock - 1) / kBlock;
    if (p.window > 0) nblk = std::min(nblk, ((long long)p.window + p.max_seqlen_q + kBlock - 1) / kBlock + 1);
    nblk = std::max(nblk, 1ll);
    const long long band = p.rel_extent > 0 ? std::min(nblk, ((long long)p.rel_extent + p.max_seqlen_q + kBlock - 1) / kBlock + 1) : 0;
    const double before = (double)(nblk - band) * kBlockUs, inside = (double)band * kI4BandCost * kBlockUs;
    const long long units = (long long)p.B * p.Hkv, slots = num_sms > 0 ? num_sms : 1;
    int best = 1;
    double best_us = 1e300;
    for (int S = 1; S <= kDecodeMaxSplits && S <= (nblk + 1) / 2; ++S) {
        double us;
        if (S == 2 && p.rel_extent > 0) {
            us = fmax(fmax((double)((units + slots - 1) / slots) * (kStart + before), kStart + inside),
                      (double)units * (2 * kStart + before + inside) / (double)slots);
        } else {
            us = (double)((units * S + slots - 1) / slots) * (kStart + (before + inside) / S);
        }
        if (S > 1) us += 2.0 + 0.27 * S + 2.0 * 4.0 * (kHeadDim + 1) * p.N_tok * (double)p.Hq * S / 6.7e6;
        if (us < best_us * (1.0 - 1e-9)) {
            best_us = us;
            best = S;
        }
    }
    return best;
}

}  // namespace

// Decode split heuristic ([vLLM TML Inkling サポート, §低レイテンシコレクティブとカーネル
// "FA4 Kernel"]: num_splits from batch size, TP size and KV length; TP = 1 here), over bf16 and E4M3 caches.
// Cost model in units of one 64-key K+V block moved at the full HBM rate: a CTA streams
// `per` blocks at min(its own rate, HBM / active CTAs), so a wave with a CTAs costs
// per * max(r, a), where r is the number of CTAs that saturate HBM; the split partials add
// their write + read traffic and the combine launch a fixed cost.
int pick_splits(const inkattn_attn_params &p, int num_sms) {
    if (p.kv_dtype == INKATTN_KV_I4) return pick_splits_i4(p, num_sms);
    const int g = p.Hq / p.Hkv;
    long long nblk = (p.max_seqlen_k + kBlock - 1) / kBlock;
    if (p.window > 0) {
        const long long span = ((long long)p.window + p.max_seqlen_q + kBlock - 1) / kBlock + 1;
        if (span < nblk) nblk = span;
    }
    if (nblk < 1) nblk = 1;
    const long long units = (long long)p.B * p.Hkv;
    const long long slots = (long long)(num_sms > 0 ? num_sms : 1) * kDecodeCtasPerSm;
    const double r = kDecodeHbmSmFrac * (double)slots;
    const long long rows_per_unit = (long long)p.max_seqlen_q * g;
    const double block_bytes = 2.0 * kBlock * kHeadDim * 2;   // K + V of one block
    // With a relative bias, two splits cut the keys at the band's start instead of halving
    // them (csrc/decode_tc.cu): the CTAs streaming the keys before the band come first in the
    // grid and the short band CTAs, whose bias tables take the longest, run beside them on
    // the SMs the last wave leaves free.  That pays when the streaming CTAs alone keep HBM
    // busy and the band is a small part of the keys; halves are then not a choice.
    const bool band_split = p.rel_extent > 0;
    const long long band_blk = ((long long)p.rel_extent + p.max_seqlen_q + kBlock - 1) / kBlock + 2;
    int best = 1;
    double best_cost = 1e300;
    for (int S = 1; S <= kDecodeMaxSplits; ++S) {
        const long long per = (nblk + S - 1) / S;
        if (S > 1 && per < kDecodeMinSplitBlocks) break;
        if (band_split && S == 2) continue;
        const long long ctas = units * S;
        const long long full = ctas / slots, rest = ctas - full * slots;
        double waves = (double)full * fmax(r, (double)slots);
        if (rest > 0) waves += fmax(r, (double)rest);
        double cost = (double)per * waves;
        if (S > 1) {
            const double ws_bytes = 2.0 * units * rows_per_unit * S * (kHeadDim + 1) * 4.0;
            cost += ws_bytes / block_bytes + kCombineCostBlocks;
        }
        if (cost < best_cost * (1.0 - 1e-9)) {
            best_cost = cost;
            best = S;
        }
    }
    if (band_split && best == 1 && (double)units >= r && nblk >= 4 * band_blk) return 2;
    return best;
}

namespace {

size_t ws_o_bytes(const inkattn_attn_params &p, int S) {
    const size_t b = (size_t)p.N_tok * p.Hq * S * kHeadDim * 4;
    return (b + 255) & ~(size_t)255;
}
size_t ws_lse_bytes(const inkattn_attn_params &p, int S) {
    const size_t b = (size_t)p.N_tok * p.Hq * S * 4;
    return (b + 255) & ~(size_t)255;
}

inkattn_status validate_decode_shape(const inkattn_attn_params &p) {
    const int g = p.Hq / p.Hkv;
    if (p.max_seqlen_q > 16 || (long long)p.max_seqlen_q * g > kDecodeMaxRows) return INKATTN_ERR_UNSUPPORTED;
    return INKATTN_OK;
}

inkattn_status resolve_splits(const inkattn_attn_params &p, int requested, int *S_out) {
    if (requested < 0 || requested > kDecodeMaxSplits) return INKATTN_ERR_INVALID_ARG;
    if (requested > 0) {
        *S_out = requested;
        return INKATTN_OK;
    }
    int sms = 0;
    inkattn_status st = check_device(&sms);
    if (st != INKATTN_OK) return st;
    *S_out = pick_splits(p, sms);
    return INKATTN_OK;
}

}  // namespace

size_t decode_workspace_bytes(const inkattn_attn_params &p, int S) {
    return S > 1 ? ws_o_bytes(p, S) + ws_lse_bytes(p, S) : 0;
}

inkattn_status validate_decode_call(const inkattn_attn_params *p, int *sms) {
    inkattn_status st = validate_attn(p);
    if (st != INKATTN_OK) return st;
    if ((st = validate_decode_shape(*p)) != INKATTN_OK) return st;
    if ((st = validate_locations(p)) != INKATTN_OK) return st;
    return check_device(sms);
}

const KernelDebug &kernel_debug() {
    static const KernelDebug d = [] {
        KernelDebug k{kWaitLimitNsDefault, 0};
        if (const char *s = std::getenv("INKATTN_TEST_WAIT_LIMIT_US")) {
            const long long us = std::atoll(s);
            if (us >= 100 && us <= 10000000) k.wait_ns = (uint64_t)us * 1000ull;
        }
        if (const char *s = std::getenv("INKATTN_TEST_WITHHOLD_ARRIVAL")) k.withhold = std::atoi(s) == 1;
        return k;
    }();
    return d;
}

bool make_cache_map(CUtensorMap *map, const void *base, long long rows) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)kHeadDim, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)kHeadDim * 2};
    cuuint32_t box[2] = {64, 64};
    cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_cache_map_e4m3(CUtensorMap *map, const void *base, long long rows) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)kHeadDim, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)kHeadDim};
    cuuint32_t box[2] = {(cuuint32_t)kHeadDim, (cuuint32_t)kBlock};
    cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_cache_map_i4(CUtensorMap *map, const void *base, long long rows) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)kHeadDim / 2, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)kHeadDim / 2};
    cuuint32_t box[2] = {(cuuint32_t)kHeadDim / 2, (cuuint32_t)kBlock};
    cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_qkvr_maps(const inkattn_qkvr_params &p, CUtensorMap *xmap, CUtensorMap *wmap) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
    if (!enc) return false;
    const long long F = (long long)(p.Hq + 2 * p.Hkv) * kHeadDim + (long long)p.Hq * p.d_r;
    cuuint64_t strides[1] = {(cuuint64_t)p.d_model * 2};
    cuuint32_t box[2] = {64, 128};
    cuuint32_t estr[2] = {1, 1};
    cuuint64_t xdims[2] = {(cuuint64_t)p.d_model, (cuuint64_t)(p.N_tok > 0 ? p.N_tok : 1)};
    cuuint64_t wdims[2] = {(cuuint64_t)p.d_model, (cuuint64_t)F};
    return enc(xmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<inkattn_bf16 *>(p.x), xdims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS &&
           enc(wmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<inkattn_bf16 *>(p.w), wdims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_linear_maps(const LinearArgs &a, bool gated, LinearMaps *maps) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
    if (!enc) return false;
    const cuuint64_t K = (cuuint64_t)a.K, F = (cuuint64_t)a.F, E = (cuuint64_t)a.E;
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    auto encode = [&](CUtensorMap *map, cuuint32_t rank, const void *base, const cuuint64_t *dims,
                      const cuuint64_t *strides, const cuuint32_t *box) {
        return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    const cuuint64_t xdims[2] = {K, (cuuint64_t)a.N_x}, xstr[1] = {K * 2};
    for (int i = 0; !a.row_token && i < a.tile_n / 32; ++i) {
        const cuuint32_t xbox[2] = {64, 16u * (cuuint32_t)(i + 1)};
        if (!encode(&maps->x[i], 2, a.x, xdims, xstr, xbox)) return false;
    }
    if (gated) {
        const cuuint64_t dims[4] = {K, F, 2, E}, str[3] = {K * 2, F * K * 2, 2 * F * K * 2};
        const cuuint32_t box[4] = {64, 64, 2, 1};
        return encode(&maps->w, 4, a.w, dims, str, box);
    }
    const cuuint64_t dims[3] = {K, F, E}, str[2] = {K * 2, F * K * 2};
    const cuuint32_t box[3] = {64, 128, 1};
    return encode(&maps->w, 3, a.w, dims, str, box);
}

bool make_q_map(CUtensorMap *map, const void *base, int n_tok, int hq, int box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)hq, (cuuint64_t)(n_tok > 0 ? n_tok : 1)};
    cuuint64_t strides[2] = {(cuuint64_t)kHeadDim * 2, (cuuint64_t)hq * kHeadDim * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_q_group_map(CUtensorMap *map, const void *base, int n_tok, int hq, int group, int tokens) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)hq, (cuuint64_t)(n_tok > 0 ? n_tok : 1)};
    cuuint64_t strides[2] = {(cuuint64_t)kHeadDim * 2, (cuuint64_t)hq * kHeadDim * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)tokens};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace inkattn

using namespace inkattn;

extern "C" {

const char *inkattn_status_string(inkattn_status s) {
    switch (s) {
        case INKATTN_OK: return "ok";
        case INKATTN_ERR_INVALID_ARG: return "invalid argument";
        case INKATTN_ERR_UNSUPPORTED: return "unsupported configuration or device";
        case INKATTN_ERR_CUDA: return "CUDA runtime error";
        case INKATTN_ERR_DEVICE_TIMEOUT: return "device wait timed out";
        case INKATTN_ERR_DEVICE_BOUNDS: return "device index out of bounds";
    }
    return "unknown status";
}

int inkattn_abi_version(void) { return INKATTN_ABI_VERSION; }

inkattn_status inkattn_prologue(const inkattn_prologue_params *p, void *stream) {
    inkattn_status st = validate_prologue(p);
    if (st != INKATTN_OK) return st;
    if ((st = check_device(nullptr)) != INKATTN_OK) return st;
    if (p->N_tok == 0) return INKATTN_OK;
    return launch_status(launch_prologue(*p, static_cast<cudaStream_t>(stream)));
}

inkattn_status inkattn_output_conv(const inkattn_output_conv_params *p, void *stream) {
    inkattn_status st = validate_output_conv(p);
    if (st != INKATTN_OK) return st;
    if ((st = check_device(nullptr)) != INKATTN_OK) return st;
    if (p->N_tok == 0) return INKATTN_OK;
    return launch_status(launch_output_conv(*p, static_cast<cudaStream_t>(stream)));
}

inkattn_status inkattn_qkvr_prologue(const inkattn_qkvr_params *p, void *stream) {
    inkattn_status st = validate_qkvr(p);
    if (st != INKATTN_OK) return st;
    int sms = 0;
    if ((st = check_device(&sms)) != INKATTN_OK) return st;
    if ((st = validate_qkvr_locations(p)) != INKATTN_OK) return st;
    // no tokens and the states in place: nothing to do
    if (p->N_tok == 0 && p->conv_state_k_out == p->conv_state_k_in && p->conv_state_v_out == p->conv_state_v_in)
        return INKATTN_OK;
    CUtensorMap xmap, wmap;
    if (!make_qkvr_maps(*p, &xmap, &wmap)) return INKATTN_ERR_CUDA;
    return launch_status(launch_qkvr(*p, xmap, wmap, sms, static_cast<cudaStream_t>(stream)));
}

inkattn_status inkattn_linear(const inkattn_linear_params *p, void *stream) {
    inkattn_status st = validate_linear(p);
    if (st != INKATTN_OK) return st;
    int sms = 0;
    if ((st = check_device(&sms)) != INKATTN_OK) return st;
    if (p->N_tok == 0) return INKATTN_OK;
    const void *read[] = {p->x, p->w};
    if ((st = validate_on_device(read, 2)) != INKATTN_OK) return st;
    LinearArgs a = {};
    a.x = p->x;
    a.w = p->w;
    a.bias = p->bias;
    a.residual = p->residual;
    a.out = p->out;
    a.dev_status = p->dev_status;
    a.E = 1;
    a.M = a.N_x = p->N_tok;
    a.K = p->K;
    a.F = p->F;
    a.out_f32 = p->out_dtype == INKATTN_DTYPE_F32;
    return launch_status(launch_linear(a, p->act, sms, static_cast<cudaStream_t>(stream)));
}

inkattn_status inkattn_grouped_linear(const inkattn_grouped_linear_params *p, void *stream) {
    inkattn_status st = validate_grouped_linear(p);
    if (st != INKATTN_OK) return st;
    int sms = 0;
    if ((st = check_device(&sms)) != INKATTN_OK) return st;
    if (p->M == 0) return INKATTN_OK;
    const void *read[] = {p->x, p->w};
    if ((st = validate_on_device(read, 2)) != INKATTN_OK) return st;
    LinearArgs a = {};
    a.x = p->x;
    a.w = p->w;
    a.bias = p->bias;
    a.out = p->out;
    a.offsets = p->expert_offsets;
    a.row_token = p->row_token;
    a.dev_status = p->dev_status;
    a.E = p->E;
    a.M = p->M;
    a.N_x = p->N_x;
    a.K = p->K;
    a.F = p->F;
    a.out_f32 = p->out_dtype == INKATTN_DTYPE_F32;
    return launch_status(launch_linear(a, p->act, sms, static_cast<cudaStream_t>(stream)));
}

size_t inkattn_route_workspace_bytes(const inkattn_route_params *p) {
    return validate_route(p, nullptr, 0) == INKATTN_OK ? route_workspace_bytes(*p) : 0;
}

inkattn_status inkattn_route(const inkattn_route_params *p, void *workspace, size_t workspace_bytes, void *stream) {
    const size_t need = inkattn_route_workspace_bytes(p);
    inkattn_status st = validate_route(p, need ? workspace : nullptr, need);
    if (st != INKATTN_OK) return st;
    if (need && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return INKATTN_ERR_INVALID_ARG;
    if ((st = check_device(nullptr)) != INKATTN_OK) return st;
    const void *read[] = {p->expert_offsets, p->N_tok > 0 ? p->logits : nullptr, workspace};
    if ((st = validate_on_device(read, need ? 3 : p->N_tok > 0 ? 2 : 1)) != INKATTN_OK) return st;
    return launch_status(launch_route(*p, static_cast<uint32_t *>(workspace), static_cast<cudaStream_t>(stream)));
}

inkattn_status inkattn_expert_combine(const inkattn_expert_combine_params *p, void *stream) {
    inkattn_status st = validate_expert_combine(p);
    if (st != INKATTN_OK) return st;
    if ((st = check_device(nullptr)) != INKATTN_OK) return st;
    if (p->N_tok == 0) return INKATTN_OK;
    const void *read[] = {p->out, p->weights};
    if ((st = validate_on_device(read, 2)) != INKATTN_OK) return st;
    return launch_status(launch_expert_combine(*p, static_cast<cudaStream_t>(stream)));
}

inkattn_status inkattn_token_probs(const inkattn_token_probs_params *p, void *stream) {
    inkattn_status st = validate_token_probs(p);
    if (st != INKATTN_OK) return st;
    int sms = 0;
    if ((st = check_device(&sms)) != INKATTN_OK) return st;
    if (p->N_tok == 0) return INKATTN_OK;
    const void *ptrs[] = {p->logits, p->probs, p->temperature};
    if ((st = validate_on_device(ptrs, p->temperature ? 3 : 2)) != INKATTN_OK) return st;
    return launch_status(launch_token_probs(*p, sms, static_cast<cudaStream_t>(stream)));
}

inkattn_status inkattn_verify_drafts(const inkattn_verify_drafts_params *p, void *stream) {
    inkattn_status st = validate_verify_drafts(p);
    if (st != INKATTN_OK) return st;
    if ((st = check_device(nullptr)) != INKATTN_OK) return st;
    // (those without rows may be NULL)
    const void *ptrs[] = {p->n_new, p->cu_seqlens_q, p->u_sample, p->target_p, p->token_ids, p->u_accept,
                          p->out_tokens, p->draft_p};
    if ((st = validate_on_device(ptrs, p->N_tok == 0 ? 3 : p->draft_p ? 8 : 7)) != INKATTN_OK) return st;
    return launch_status(launch_verify_drafts(*p, static_cast<cudaStream_t>(stream)));
}

inkattn_status inkattn_conv_rollback(const inkattn_conv_rollback_params *p, void *stream) {
    inkattn_status st = validate_conv_rollback(p);
    if (st != INKATTN_OK) return st;
    if ((st = check_device(nullptr)) != INKATTN_OK) return st;
    const void *ptrs[3 + 3 * INKATTN_ROLLBACK_MAX_STATES] = {p->cu_seqlens_q, p->state_slot, p->n_keep};
    int n = 3;
    for (int s = 0; s < p->n_states; ++s) {
        const inkattn_conv_rows &c = p->states[s];
        if (p->N_tok > 0) ptrs[n++] = c.x;             // (may be NULL without rows)
        ptrs[n++] = c.state_before;
        if (c.state_after != c.state_before) ptrs[n++] = c.state_after;
    }
    if ((st = validate_on_device(ptrs, n)) != INKATTN_OK) return st;
    return launch_status(launch_conv_rollback(*p, static_cast<cudaStream_t>(stream)));
}

namespace {

// The prefill over a bf16 cache, once the call is validated.
inkattn_status run_prefill_bf16(const inkattn_attn_params &p, cudaStream_t stream) {
    CUtensorMap qmap, kmap, vmap;
    const long long rows = (long long)p.num_blocks * p.Hkv * kBlock;
    if (!make_q_map(&qmap, p.q, p.N_tok, p.Hq, kPrefillTcRows) ||
        !make_cache_map(&kmap, p.k_cache, rows) || !make_cache_map(&vmap, p.v_cache, rows))
        return INKATTN_ERR_CUDA;
    if (p.rel_extent == 0)   // no bias band: two query tiles per CTA
        return launch_status(launch_prefill_2q(p, scalars(p), qmap, kmap, vmap, stream));
    return launch_status(launch_prefill_tc(p, scalars(p), qmap, kmap, vmap, stream));
}

// Workspace of the prefill over a cache of codes: bf16 K and V copies of B * max_blocks_per_seq
// blocks, then their block table, each piece 256-byte aligned.
size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }
size_t prefill_copy_bytes(const inkattn_attn_params &p) {
    return (size_t)p.B * p.max_blocks_per_seq * p.Hkv * kBlock * kHeadDim * 2;
}
size_t prefill_ws_bytes(const inkattn_attn_params &p) {
    return 2 * round256(prefill_copy_bytes(p)) + round256((size_t)p.B * p.max_blocks_per_seq * 4);
}

}  // namespace

inkattn_status inkattn_prefill(const inkattn_attn_params *p, void *stream) {
    inkattn_status st = validate_attn(p);
    if (st != INKATTN_OK) return st;
    if (p->kv_dtype != INKATTN_KV_BF16) return INKATTN_ERR_UNSUPPORTED;   // (inkattn_prefill_e4m3, _i4)
    if ((st = validate_locations(p)) != INKATTN_OK) return st;
    if ((st = check_device(nullptr)) != INKATTN_OK) return st;
    if (p->N_tok == 0) return INKATTN_OK;
    return run_prefill_bf16(*p, static_cast<cudaStream_t>(stream));
}

size_t inkattn_prefill_workspace_bytes(const inkattn_attn_params *p) {
    if (validate_attn(p) != INKATTN_OK || p->kv_dtype == INKATTN_KV_BF16) return 0;
    return prefill_ws_bytes(*p);
}

// The prefill over a cache of codes of the given type.
static inkattn_status prefill_codes(const inkattn_attn_params *p, int32_t kv_dtype, void *workspace,
                                    size_t workspace_bytes, void *stream) {
    inkattn_status st = validate_attn(p);
    if (st != INKATTN_OK) return st;
    if (p->kv_dtype != kv_dtype) return INKATTN_ERR_INVALID_ARG;
    // the copy's rows are addressed by TMA as 32-bit coordinates
    if ((long long)p->B * p->max_blocks_per_seq * p->Hkv * kBlock >= (1ll << 31)) return INKATTN_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < prefill_ws_bytes(*p))
        return INKATTN_ERR_INVALID_ARG;
    if ((st = check_device(nullptr)) != INKATTN_OK) return st;
    if ((st = validate_locations(p)) != INKATTN_OK) return st;
    {   // the copy is read by TMA too: device memory of this GPU
        int dev = -1;
        cudaPointerAttributes a;
        if (cudaGetDevice(&dev) != cudaSuccess || cudaPointerGetAttributes(&a, workspace) != cudaSuccess) {
            (void)cudaGetLastError();
            return INKATTN_ERR_INVALID_ARG;
        }
        if (a.type != cudaMemoryTypeDevice || a.device != dev) return INKATTN_ERR_INVALID_ARG;
    }
    if (p->N_tok == 0) return INKATTN_OK;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    const size_t copy = round256(prefill_copy_bytes(*p));
    inkattn_bf16 *k16 = reinterpret_cast<inkattn_bf16 *>(ws);
    inkattn_bf16 *v16 = reinterpret_cast<inkattn_bf16 *>(ws + copy);
    int32_t *table = reinterpret_cast<int32_t *>(ws + 2 * copy);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((st = launch_status(launch_dequant(*p, k16, v16, table, s))) != INKATTN_OK) return st;
    inkattn_attn_params q = *p;
    q.k_cache = k16;
    q.v_cache = v16;
    q.kv_dtype = INKATTN_KV_BF16;
    q.k_scale = nullptr;
    q.v_scale = nullptr;
    q.block_table = table;
    q.num_blocks = p->B * p->max_blocks_per_seq;
    return run_prefill_bf16(q, s);
}

inkattn_status inkattn_prefill_e4m3(const inkattn_attn_params *p, void *workspace, size_t workspace_bytes,
                                    void *stream) {
    return prefill_codes(p, INKATTN_KV_E4M3, workspace, workspace_bytes, stream);
}

inkattn_status inkattn_prefill_i4(const inkattn_attn_params *p, void *workspace, size_t workspace_bytes, void *stream) {
    return prefill_codes(p, INKATTN_KV_I4, workspace, workspace_bytes, stream);
}

int inkattn_decode_num_splits(const inkattn_attn_params *p, int num_sms) {
    if (validate_attn(p) != INKATTN_OK || validate_decode_shape(*p) != INKATTN_OK || num_sms < 1) return 0;
    return pick_splits(*p, num_sms);
}

size_t inkattn_decode_workspace_bytes(const inkattn_attn_params *p, int num_splits) {
    if (validate_attn(p) != INKATTN_OK) return 0;
    int S = 0;
    if (resolve_splits(*p, num_splits, &S) != INKATTN_OK || S <= 1) return 0;
    return ws_o_bytes(*p, S) + ws_lse_bytes(*p, S);
}

inkattn_status inkattn_decode(const inkattn_attn_params *p, int num_splits, void *workspace,
                              size_t workspace_bytes, void *stream) {
    inkattn_status st = validate_attn(p);
    if (st != INKATTN_OK) return st;
    if ((st = validate_decode_shape(*p)) != INKATTN_OK) return st;
    if (num_splits < 0 || num_splits > kDecodeMaxSplits) return INKATTN_ERR_INVALID_ARG;
    if ((st = validate_locations(p)) != INKATTN_OK) return st;
    if ((st = check_device(nullptr)) != INKATTN_OK) return st;
    int S = 0;
    if ((st = resolve_splits(*p, num_splits, &S)) != INKATTN_OK) return st;
    float *ws_o = nullptr, *ws_lse = nullptr;
    if (S > 1) {
        const size_t need = ws_o_bytes(*p, S) + ws_lse_bytes(*p, S);
        if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return INKATTN_ERR_INVALID_ARG;
        ws_o = static_cast<float *>(workspace);
        ws_lse = reinterpret_cast<float *>(static_cast<char *>(workspace) + ws_o_bytes(*p, S));
    }
    if (p->N_tok == 0) return INKATTN_OK;
    CUtensorMap qmap, kmap, vmap;
    const long long rows = (long long)p->num_blocks * p->Hkv * kBlock;
    auto cache_map = p->kv_dtype == INKATTN_KV_I4     ? make_cache_map_i4
                     : p->kv_dtype == INKATTN_KV_E4M3 ? make_cache_map_e4m3
                                                      : make_cache_map;
    if (!cache_map(&kmap, p->k_cache, rows) || !cache_map(&vmap, p->v_cache, rows) ||
        !make_q_group_map(&qmap, p->q, p->N_tok, p->Hq, p->Hq / p->Hkv, p->max_seqlen_q))
        return INKATTN_ERR_CUDA;
    return launch_status(launch_decode_tc(*p, scalars(*p), S, ws_o, ws_lse, qmap, kmap, vmap,
                                          static_cast<cudaStream_t>(stream)));
}

inkattn_status inkattn_combine(const inkattn_attn_params *p, int num_splits, const void *workspace,
                               size_t workspace_bytes, void *stream) {
    inkattn_status st = validate_attn(p);
    if (st != INKATTN_OK) return st;
    if ((st = validate_decode_shape(*p)) != INKATTN_OK) return st;
    if (num_splits < 0 || num_splits > kDecodeMaxSplits) return INKATTN_ERR_INVALID_ARG;
    if ((st = check_device(nullptr)) != INKATTN_OK) return st;
    int S = 0;
    if ((st = resolve_splits(*p, num_splits, &S)) != INKATTN_OK) return st;
    if (S <= 1 || p->N_tok == 0) return INKATTN_OK;
    const size_t need = ws_o_bytes(*p, S) + ws_lse_bytes(*p, S);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return INKATTN_ERR_INVALID_ARG;
    const float *ws_o = static_cast<const float *>(workspace);
    const float *ws_lse = reinterpret_cast<const float *>(static_cast<const char *>(workspace) + ws_o_bytes(*p, S));
    return launch_status(launch_combine(*p, S, ws_o, ws_lse, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
