// rollback.cu -- conv states of the tokens that a verification step kept.
//
// [vLLM hỗ trợ TML Inkling ..., §Quản lý bộ nhớ đệm sconv]: the state keeps the hidden states of the
// last W - 1 = 3 tokens; a step over a sequence's last token and its drafts leaves the state of
// all of them, and the rejected ones have to leave it again.
//
// With xs = the 3 rows of the state before the step, then the step's rows of the conv's input, the
// state behind the first n rows is xs[n .. n + 2].  A thread takes 8 channels of one sequence and
// conv: it reads the three 16-byte pieces and then writes them, so the states may be updated in place.
// One launch for all the convs of a layer (K, V, attention output, MLP output): a sequence moves 6 bytes a
// channel in and 6 out, so four launches would cost little else (one sequence of 18432 channels
// 3.9 us, the launch; 512 sequences 18.8 us, 6.0 TB/s).
#include "common.cuh"
#include "internal.h"

namespace inkattn {

namespace {
constexpr int kRollbackThreads = 128;      // 8 channels each
}

__global__ void __launch_bounds__(kRollbackThreads)
k_conv_rollback(const inkattn_conv_rollback_params p) {
    grid_dep_wait();
    grid_dep_launch();
    // which conv, and which of its pieces
    int part = blockIdx.x, s = 0;
    int parts = (p.states[0].C / 8 + kRollbackThreads - 1) / kRollbackThreads;
    while (part >= parts) {                // (the grid holds the sum of the parts)
        part -= parts;
        ++s;
        parts = (p.states[s].C / 8 + kRollbackThreads - 1) / kRollbackThreads;
    }
    const inkattn_conv_rows &c = p.states[s];
    const int b = blockIdx.y;
    const int start = load_i32(p.cu_seqlens_q + b), end = load_i32(p.cu_seqlens_q + b + 1);
    const int slot = load_i32(p.state_slot + b), n = load_i32(p.n_keep + b);
    if (start < 0 || end < start || end > p.N_tok || slot < 0 || slot >= p.num_state_slots || n < 0 ||
        n > end - start) {
        if (threadIdx.x == 0) set_status(p.dev_status, INKATTN_ERR_DEVICE_BOUNDS);
        return;
    }
    const int ch = (part * kRollbackThreads + threadIdx.x) * 8;
    if (ch >= c.C) return;
    const size_t st = (size_t)slot * 3 * c.C + ch;
    uint4 v[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int at = n + i - 3;          // place among the step's rows; below 0 the old state's
        v[i] = at < 0 ? load_u32x4(c.state_before + st + (size_t)(at + 3) * c.C)
                      : load_u32x4(c.x + (size_t)(start + at) * c.x_stride + ch);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) *reinterpret_cast<uint4 *>(c.state_after + st + (size_t)i * c.C) = v[i];
}

cudaError_t launch_conv_rollback(const inkattn_conv_rollback_params &p, cudaStream_t stream) {
    int parts = 0;
    for (int s = 0; s < p.n_states; ++s) parts += (p.states[s].C / 8 + kRollbackThreads - 1) / kRollbackThreads;
    return launch_dependent(k_conv_rollback, dim3(parts, p.B), dim3(kRollbackThreads), 0, stream, 1, p);
}

}  // namespace inkattn
