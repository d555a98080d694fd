// paged.h -- launch arguments of the paged-cache operators.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace fa {

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
    int shift;  // log2(page_size)
};

// Division of x < 2^31 by a fixed d >= 1 as a multiplication: with s the
// smallest such that 2^s >= d and mul = floor(2^32 (2^s - d) / d) + 1,
// x / d = (hi32(x mul) + x) >> s  (Granlund and Montgomery, 1994).
struct FastDiv {
    uint32_t mul;
    int shift, d;
};

inline FastDiv fast_div(int d) {
    FastDiv f{0, 0, d};
    while ((1ll << f.shift) < d) ++f.shift;
    f.mul = (uint32_t)(((1ull << 32) * ((1ull << f.shift) - d)) / d + 1);
    return f;
}

// Where the partial results of one pass over keys (the shared prefix', or the
// requests' own) lie.  A pass gives every row one result, or several where
// CTAs shared the row's keys.  Each is O~ / l in fp32 and lse2, log2 of the
// sum of exponentials (-inf: nothing seen); several merge as
//   O = sum w_i O_i / sum w_i,  w_i = 2^(lse2_i - max).
// code[row] says which a row has (row = token * Hq + head): 0 one, final or in
// the plane; otherwise pieces | first CTA << 9 | row within the slot << 18 |
// kFewCode: slot 1 of the first CTA and slot 0 of the following ones, the
// few-row kernel's where both kernels share the own pass.
struct PartView {
    int *code;                  // [total * Hq]
    float *plane_lse2, *plane;  // [total * Hq] (x d); null where one result is final
    float *slot_lse2, *slot;    // [ctas][2][slot_rows] (x d)
    float *slot_sum;            // 256-row kernel: of a row that is being worked on (slot_lse2: its maximum)
    int slot_rows, ctas;
};
constexpr int kSms = 152;  // of the GPU; the workspace's size must not depend on a query
constexpr int kMaxRows = 16;  // rows of a (request, key/value head) pair in the few-row kernel
constexpr int kWideRows = 256, kWideKeys = 128;  // row block and key tile of the 256-row kernel
constexpr int kMaxPieces = 511;  // 9 bits, also of CTA numbers

constexpr int kFewCode = 1 << 26;

__host__ __device__ constexpr int part_code(int pieces, int cta, int row) { return pieces | cta << 9 | row << 18; }

// How a call is divided among the kernels.
struct PagedPlan {
    bool few;         // own keys by the 16-row kernel, else by the 256-row one
    bool joined;      // the shared prefix' keys too, with each request's own
    bool mixed;       // by both: requests of at most 16 rows (a pair) by the first
    bool whole;       // the 16-row kernel's CTAs take whole pairs only: nothing to merge
    long long own_tiles, prefix_tiles;  // key tiles of a row block of the 256-row kernel, at most
    PartView own;     // ctas: of the kernel that takes the own keys
    PartView beside;  // mixed: of the 16-row kernel; codes and planes are own's
    PartView prefix;  // ctas 0: no pass over a shared prefix
    size_t bytes;     // workspace
};

// The workspace needed is the largest without a window.
PagedPlan plan_paged(int B, int total, int max_new, int Hq, int Hkv, int d, int max_pages, int page_size,
                     int prefix_len, int window, void *workspace);

// The kernels of a forward call.  `after`: beside the call's kernel before.
cudaError_t launch_paged_few(const PagedArgs &a, const PagedPlan &w, bool after, cudaStream_t st);
cudaError_t launch_paged_wide(const PagedArgs &a, const PagedPlan &w, bool prefix, bool after, cudaStream_t st);
cudaError_t launch_paged_merge(const PagedArgs &a, const PagedPlan &w, cudaStream_t st);

cudaError_t launch_paged_tables(const TablesArgs &a, cudaStream_t st);
cudaError_t launch_paged_append(const AppendArgs &a, cudaStream_t st);
cudaError_t launch_fwd_paged(const PagedArgs &a, cudaStream_t st);

}  // namespace fa
