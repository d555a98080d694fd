// paged.h -- launch arguments of the paged-cache operators.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace fa {

// Requests one fa_paged_tables call takes: every block keeps two 32-bit
// prefix sums per request in shared memory (128 KB of the 227 KB).
constexpr int kMaxTableRequests = 16384;

struct TablesArgs {
    const int *cached_lens, *new_lens, *free_pages, *free_start;
    int *block_table, *seq_lens, *cu_seqlens, *slots, *counts;
    int B, max_pages, page_size, num_pages, num_free, total;
};

struct AppendArgs {
    const void *k, *v;
    const int *slots;
    void *k_cache, *v_cache;
    int total, Hkv, d, page_size, num_pages;
};

struct PagedArgs {
    const void *q, *k_cache, *v_cache;
    const int *block_table, *seq_lens;
    const int *cu_seqlens;    // null: one row per request
    const int *prefix_pages;  // null without a shared prefix
    void *o;
    float *lse;
    int B, total, max_new, Hq, Hkv, d;
    int max_pages, page_size, num_pages;
    int prefix_len;  // 0: no shared prefix
    int window;      // 0: none
    float scale;
    bool bf16;
    void *workspace;
};

// How a call is divided for the 256-row kernel (fa_fwd_paged_wide.cu): row
// blocks (upper bounds, the real ones depend on the device's offsets) and key
// ranges per block, for the shared prefix and for the requests' own keys; 0
// ranges: not this kernel's.  Partial results are planes [range][total][Hq],
// the prefix' first.
struct WidePlan {
    int prefix_blocks, prefix_splits;
    int own_blocks, own_splits;
    float *part_o, *part_lse2;
};

cudaError_t launch_paged_wide(const PagedArgs &a, int shift, const WidePlan &w, cudaStream_t st);

cudaError_t launch_paged_tables(const TablesArgs &a, cudaStream_t st);
cudaError_t launch_paged_append(const AppendArgs &a, cudaStream_t st);
cudaError_t launch_fwd_paged(const PagedArgs &a, cudaStream_t st);
// Workspace bytes of launch_fwd_paged (shapes only, no device query).
size_t fwd_paged_workspace(int B, int total, int max_new, int Hq, int Hkv, int d, int max_pages, int page_size,
                           int prefix_len);

}  // namespace fa
