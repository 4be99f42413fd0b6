// Order among the calls of a context that share its workspace.
#pragma once

#include <cuda_runtime.h>

namespace domino {

// The workspace's last user: outside of graph capture, and in the capture `captured_id` (0: none).
struct WorkspaceUse {
    cudaEvent_t used, captured;
    bool was_used;
    unsigned long long captured_id;

    cudaError_t create() {
        const cudaError_t e = cudaEventCreateWithFlags(&used, cudaEventDisableTiming);
        return e == cudaSuccess ? cudaEventCreateWithFlags(&captured, cudaEventDisableTiming) : e;
    }
    void release() {
        if (used) cudaEventDestroy(used);
        if (captured) cudaEventDestroy(captured);
    }
};

// Orders the calls that use the workspace among each other, whatever their
// streams: a call waits for the event that the last one recorded.  Always, even
// on what looks like the same stream: a handle's value may be another stream's by
// now.  An event recorded outside of a capture cannot be waited for inside it, nor
// the other way round, so a capture has an event of its own for its calls.
struct WorkspaceOrder {
    WorkspaceUse* use;
    cudaStream_t st;
    bool capturing = false;
    cudaError_t error;

    WorkspaceOrder(WorkspaceUse* use_, cudaStream_t st_) : use(use_), st(st_) {
        cudaStreamCaptureStatus status;
        unsigned long long id = 0;
        error = cudaStreamGetCaptureInfo(st, &status, &id);
        if (error != cudaSuccess) return;
        capturing = status == cudaStreamCaptureStatusActive;
        if (capturing) {
            if (use->captured_id == id) error = cudaStreamWaitEvent(st, use->captured, 0);
            use->captured_id = id;
        } else if (use->was_used) {
            error = cudaStreamWaitEvent(st, use->used, 0);
        }
    }
    // after the launches, also where one of them failed
    cudaError_t done() {
        if (!capturing) use->was_used = true;
        return cudaEventRecord(capturing ? use->captured : use->used, st);
    }
};

}  // namespace domino
