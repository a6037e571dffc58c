// Helpers of the host layer shared by the C entry points (ttt_api.cu, ttt_block_api.cu):
// alignment and overlap checks, and the status of a launch.
#pragma once

#include <cstdint>
#include <cstdlib>
#include <cstring>

#include "block_internal.h"

namespace ttt {

struct Span {
    const void* p;
    size_t bytes;
};

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool overlap(Span a, Span b) {
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

inline bool check_env() {
    static const bool on = [] {
        const char* v = std::getenv("TTT_CHECK");
        return v && v[0] && std::strcmp(v, "0") != 0;
    }();
    // the fault-injection hook makes a launch abandon its waits: report that as a status
    return on || drop_chunk_hook() >= 0;
}

// In check mode the device error words are cleared before the launch, so the
// status a checked call returns reflects that call alone (calls overlapping on
// several streams still share the words).
inline bool prepare() {
    if (!check_env()) return true;
    unsigned int stale = 0;
    return read_and_clear_device_error(&stale) == cudaSuccess &&
           read_and_clear_mlp_error(&stale) == cudaSuccess &&
           read_and_clear_umma_error(&stale) == cudaSuccess &&
           read_and_clear_prologue_error(&stale) == cudaSuccess &&
           read_and_clear_prologue_q8_error(&stale) == cudaSuccess;
}

// Outputs must not overlap any other buffer, except that an output state
// buffer may be exactly its initial-state buffer (in-place update).
inline ttt_status check_aliasing(const Span* outs, int n_out, const Span* ins, const int* same_as, int n_in) {
    for (int o = 0; o < n_out; o++) {
        for (int i = 0; i < n_in; i++) {
            if (same_as[o] == i && outs[o].p == ins[i].p) continue;
            if (overlap(outs[o], ins[i])) return TTT_ERR_ALIAS;
        }
        for (int o2 = o + 1; o2 < n_out; o2++)
            if (overlap(outs[o], outs[o2])) return TTT_ERR_ALIAS;
    }
    return TTT_OK;
}

inline ttt_status finish(cudaError_t launch, cudaStream_t stream) {
    if (launch != cudaSuccess) return TTT_ERR_CUDA;
    if (!check_env()) return TTT_OK;
    if (cudaStreamSynchronize(stream) != cudaSuccess) return TTT_ERR_CUDA;
    unsigned int flag = 0, mlp_flag = 0, umma_flag = 0, pro_flag = 0, q8_flag = 0;
    if (read_and_clear_device_error(&flag) != cudaSuccess) return TTT_ERR_CUDA;
    if (read_and_clear_mlp_error(&mlp_flag) != cudaSuccess) return TTT_ERR_CUDA;
    if (read_and_clear_umma_error(&umma_flag) != cudaSuccess) return TTT_ERR_CUDA;
    if (read_and_clear_prologue_error(&pro_flag) != cudaSuccess) return TTT_ERR_CUDA;
    if (read_and_clear_prologue_q8_error(&q8_flag) != cudaSuccess) return TTT_ERR_CUDA;
    return (flag | mlp_flag | umma_flag | pro_flag | q8_flag) ? TTT_ERR_TIMEOUT : TTT_OK;
}

}  // namespace ttt
