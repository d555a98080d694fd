// paged_dev.cuh -- device-side pieces shared by the paged forward kernels.
#pragma once

#include "paged.h"
#include "status.cuh"

namespace fa {

// A request as the kernels see it: its rows are row0 .. row0 + n - 1 of q and
// its own keys 0 .. len - 1.
struct Request {
    int row0, n, len;
};

// False if what the device holds for request b breaks the rules of the call
// (offsets, row bound, length): it then has no rows.
__device__ __forceinline__ bool load_request(const PagedArgs &a, int b, Request &r) {
    r.row0 = b;
    r.n = 1;
    if (a.cu_seqlens) {
        r.row0 = a.cu_seqlens[b];
        const int end = a.cu_seqlens[b + 1];
        if (r.row0 < 0 || end < r.row0 || end > a.total || end - r.row0 > a.max_new) return false;
        r.n = end - r.row0;
    }
    r.len = a.seq_lens[b];
    return r.len >= 0 && r.len <= (a.max_pages << a.shift);
}

// Programmatic dependent launch: lets the stream's next kernel start as soon
// as every CTA of this one has started, and waits until the kernel before
// this one has finished and its writes are visible.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace fa
