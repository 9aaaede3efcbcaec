// host.h -- what every translation unit's host side shares: the calling thread's failure
// record (swiglu_mlp_last_error_detail), its launch trace (swiglu_mlp_trace_begin) and the
// device's SM count.  Defined in swiglu_mlp.cu.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "swiglu_mlp.h"

namespace swiglu {

struct Trace {
    cudaEvent_t* events = nullptr;
    int* kinds = nullptr;
    int capacity = 0;
    int count = 0;
};
extern thread_local Trace g_trace;

// Records what failed on this thread and returns `st`.
swiglu_status fail(swiglu_status st, const char* what, cudaError_t err = cudaSuccess);

// SM count of the current device (whose primary context becomes current).
swiglu_status device_sms(int* num_sms);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// One kernel launch, bracketed by the launch trace's events when one is open.
template <class F>
swiglu_status launch_traced(int kind, cudaStream_t stream, F&& do_launch) {
    Trace& tr = g_trace;
    const int slot = tr.events ? tr.count++ : -1;
    const bool traced = slot >= 0 && slot < tr.capacity;
    cudaError_t e;
    if (traced) {
        tr.kinds[slot] = kind;
        e = cudaEventRecord(tr.events[2 * slot], stream);
        if (e != cudaSuccess) return fail(SWIGLU_ERR_CUDA, "cudaEventRecord(trace)", e);
    }
    e = do_launch();
    if (e != cudaSuccess) return fail(SWIGLU_ERR_LAUNCH, "kernel launch", e);
    if (traced) {
        e = cudaEventRecord(tr.events[2 * slot + 1], stream);
        if (e != cudaSuccess) return fail(SWIGLU_ERR_CUDA, "cudaEventRecord(trace)", e);
    }
    return SWIGLU_OK;
}

}  // namespace swiglu
