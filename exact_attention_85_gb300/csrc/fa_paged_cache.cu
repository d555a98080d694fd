// fa_paged_cache.cu -- the bookkeeping and the writes of a paged key/value
// cache: pages and slots for new tokens (fa_paged_tables), and the copy of
// their keys and values into those slots (fa_paged_append).
#include "../../include/fa.h"
#include "host_util.h"
#include "paged.h"
#include "paged_dev.cuh"
#include "status.cuh"

#include <algorithm>

namespace fa {

namespace {

constexpr int kTabThreads = 256;

struct TablesParams {
    TablesArgs a;
    int shift;  // log2(page_size)
    unsigned int *status;
};

__device__ __forceinline__ int pages_of(long long tokens, int shift) {
    return (int)((tokens + (1ll << shift) - 1) >> shift);
}

// A request's lengths as they count: both non-negative, their sum within the
// table's row.  A request that breaks this gets no rows and no pages.
__device__ __forceinline__ bool request_lens(const TablesParams &p, int b, int &cached, int &fresh) {
    cached = p.a.cached_lens[b];
    fresh = p.a.new_lens[b];
    if (cached >= 0 && fresh >= 0 && (long long)cached + fresh <= ((long long)p.a.max_pages << p.shift)) return true;
    cached = 0;
    fresh = 0;
    return false;
}

// Pages and slots in one launch.  Request b needs
//   need_b = ceil((c_b + n_b) / ps) - ceil(c_b / ps)
// pages and takes those at first_b = sum of the needs before it in the free
// list; its new rows start at cu_b = sum of the n before it.  Both sums run
// over all requests, and every slot needs both.  A launch of its own for the
// sums would cost more than the sums: so every block forms them for itself
// (two integers a request, read from L2) and then writes its share of the
// outputs: requests, handed-out pages and rows, each dealt over all threads of
// the grid, the request of a page or a row looked up by bisection in shared
// memory.  No block waits for another: a slot in a page that this call hands
// out takes the page from the free list, not from the table cell another
// thread writes.  Bound by latency, not by its bytes: lengths, then pages,
// then stores (one new token each for 8 requests 2.4 us, for 1024 4.0, 16384
// 14; one prompt of 500 thousand tokens 4.3).  R: consecutive rows a thread; four (one store, and often one
// page) where there are rows for every SM's threads, else one.
template <int R>
__global__ void __launch_bounds__(kTabThreads) paged_tables_kernel(const TablesParams p) {
    extern __shared__ int smem[];
    const int B = p.a.B;
    int *cu = smem;             // [B + 1], clipped to total
    int *first = smem + B + 1;  // [B], saturated
    int *held = first + B;      // [B], cached lengths
    __shared__ long long warp_rows[kTabThreads / 32], warp_need[kTabThreads / 32];
    __shared__ int taken;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (B + kTabThreads - 1) / kTabThreads | 1;  // odd: neighbouring threads in different banks
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);

    wait_previous();
    launch_dependents();
    const int start_in = p.a.free_start ? *p.a.free_start : 0;
    const bool start_ok = start_in >= 0 && start_in <= p.a.num_free;
    const int start = start_ok ? start_in : 0;
    const int room = start_ok ? p.a.num_free - start : 0;

    bool bad = !start_ok;
#pragma unroll 4
    for (int b = tid; b < B; b += kTabThreads) {
        int c, n;
        if (!request_lens(p, b, c, n)) bad = true;
        held[b] = c;
        cu[b] = n;
    }
    __syncthreads();
    auto pages_needed = [&](int c, int n) {
        return pages_of((long long)c + n, p.shift) - pages_of(c, p.shift);
    };
    long long rows = 0, need = 0;
    for (int b = b0; b < b1; ++b) {
        rows += cu[b];
        need += pages_needed(held[b], cu[b]);
    }
    // exclusive sums over the threads: within the warp, then over the warps
    long long r_in = rows, n_in = need;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const long long r = __shfl_up_sync(0xffffffffu, r_in, s), n = __shfl_up_sync(0xffffffffu, n_in, s);
        if (lane >= s) {
            r_in += r;
            n_in += n;
        }
    }
    if (lane == 31) {
        warp_rows[warp] = r_in;
        warp_need[warp] = n_in;
    }
    if (tid == 0) taken = 0x7FFFFFFF;
    __syncthreads();
    long long r_at = r_in - rows, n_at = n_in - need, r_all = 0, n_all = 0;
#pragma unroll
    for (int w = 0; w < kTabThreads / 32; ++w) {
        if (w < warp) {
            r_at += warp_rows[w];
            n_at += warp_need[w];
        }
        r_all += warp_rows[w];
        n_all += warp_need[w];
    }
    if (r_all > p.a.total) bad = true;
    for (int b = b0; b < b1; ++b) {
        const int n = cu[b], nd = pages_needed(held[b], n);
        cu[b] = (int)min(r_at, (long long)p.a.total);
        first[b] = (int)min(n_at, 0x7FFFFFFFll);
        // the first request that does not fit ends what is taken
        if (nd > 0 && n_at + nd > room) atomicMin(&taken, first[b]);
        r_at += n;
        n_at += nd;
    }
    if (tid == 0) cu[B] = (int)min(r_all, (long long)p.a.total);
    __syncthreads();
    if (bad && blockIdx.x == 0) record_bad_args(p.status);

    if (blockIdx.x == 0 && tid == 0) {
        const bool all = n_all <= room;
        p.a.counts[0] = start + (all ? (int)n_all : taken);
        p.a.counts[1] = all ? 0 : (int)min(n_all - room, 0x7FFFFFFFll);
        p.a.cu_seqlens[B] = cu[B];
    }
    // the last of the requests whose entry (of cu or first) is at most x
    auto find = [&](const int *at, int x) {
        int lo = 0, hi = B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (at[mid] <= x) lo = mid; else hi = mid - 1;
        }
        return lo;
    };
    const long long id = (long long)blockIdx.x * kTabThreads + tid, threads = (long long)gridDim.x * kTabThreads;
    for (long long b = id; b < B; b += threads) {
        const int c = held[b], n = cu[b + 1] - cu[b];
        const int nd = pages_needed(c, n);
        p.a.seq_lens[b] = nd == 0 || (long long)first[b] + nd <= room ? c + n : c;
        p.a.cu_seqlens[b] = cu[b];
    }
    // table cells, by the page's place in the free list
    const int handed = (int)min(n_all, (long long)min(taken, room));
    for (long long i = id; i < handed; i += threads) {
        const int page = p.a.free_pages[start + i];
        if (page < 0 || page >= p.a.num_pages) record_bad_args(p.status);
        const int b = find(first, (int)i), c = held[b];
        const int k = (int)i - first[b];
        if (k < pages_needed(c, cu[b + 1] - cu[b]))
            p.a.block_table[(size_t)b * p.a.max_pages + pages_of(c, p.shift) + k] = page;
    }
    // slots
    for (long long r0 = id * R; r0 < p.a.total; r0 += threads * R) {
        int out[R];
        int b = -1, c = 0, old = 0, page_at = -1, page = -1;
        bool served = false;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int r = (int)min(r0 + k, (long long)0x7FFFFFFE);
            out[k] = -1;
            if (r >= cu[B]) continue;
            if (b < 0 || r >= cu[b + 1]) {
                b = find(cu, r);
                c = held[b];
                old = pages_of(c, p.shift);
                const int nd = pages_needed(c, cu[b + 1] - cu[b]);
                served = nd == 0 || (long long)first[b] + nd <= room;
                page_at = -1;
            }
            if (!served) continue;
            const int at = c + (r - cu[b]);
            const int pg = at >> p.shift;
            if (pg != page_at) {
                page = pg < old ? p.a.block_table[(size_t)b * p.a.max_pages + pg]
                                : p.a.free_pages[start + first[b] + pg - old];
                if (page < 0 || page >= p.a.num_pages) {
                    record_bad_args(p.status);
                    page = -1;
                }
                page_at = pg;
            }
            if (page >= 0) out[k] = (page << p.shift) + (at & ((1 << p.shift) - 1));
        }
        if (R == 4 && r0 + 4 <= p.a.total) {
            *reinterpret_cast<int4 *>(p.a.slots + r0) = make_int4(out[0], out[1 % R], out[2 % R], out[3 % R]);
        } else {
#pragma unroll
            for (int k = 0; k < R; ++k)
                if (r0 + k < p.a.total) p.a.slots[r0 + k] = out[k];
        }
    }
}

// ------------------------------------------------------------------ append

constexpr int kAppThreads = 256;

struct AppendParams {
    AppendArgs a;
    FastDiv chunks;    // 16-byte pieces of one row: Hkv * d / 8
    FastDiv d_chunks;  // of one head: d / 8
    int rows_per_block;
    int shift;  // log2(page_size)
    unsigned int *status;
};

// 16-byte pieces of k and v; the destination row comes from slots[].
// [total][Hkv][d] -> [page][Hkv][ps][d]: a (row, head) piece of d values is
// contiguous on both sides.  A copy: bound by memory, so every thread has four
// pieces of k and of v in flight at a time.
constexpr int kAppUnroll = 4;

__global__ void __launch_bounds__(kAppThreads) paged_append_kernel(const AppendParams p) {
    const int row0 = blockIdx.x * p.rows_per_block;
    const int rows = min(p.rows_per_block, p.a.total - row0);
    const uint4 *k = static_cast<const uint4 *>(p.a.k) + (size_t)row0 * p.chunks.d;
    const uint4 *v = static_cast<const uint4 *>(p.a.v) + (size_t)row0 * p.chunks.d;
    uint4 *kc = static_cast<uint4 *>(p.a.k_cache), *vc = static_cast<uint4 *>(p.a.v_cache);
    const int limit = p.a.num_pages << p.shift, pieces = rows * p.chunks.d;
    wait_previous();
    launch_dependents();
    for (int i0 = threadIdx.x; i0 < pieces; i0 += kAppThreads * kAppUnroll) {
        size_t to[kAppUnroll];
        uint4 x[kAppUnroll], y[kAppUnroll];
        bool live[kAppUnroll];
#pragma unroll
        for (int j = 0; j < kAppUnroll; ++j) {
            const int i = i0 + j * kAppThreads;
            live[j] = i < pieces;
            if (!live[j]) continue;
            const int row = i / p.chunks, rest = i - row * p.chunks.d;
            const int slot = p.a.slots[row0 + row];
            const int h = rest / p.d_chunks, c = rest - h * p.d_chunks.d;
            x[j] = __ldcs(k + i);
            y[j] = __ldcs(v + i);
            live[j] = slot >= 0 && slot < limit;
            if (slot >= limit) record_bad_args(p.status);
            to[j] = ((((size_t)(slot >> p.shift) * p.a.Hkv + h) << p.shift) + (slot & ((1 << p.shift) - 1))) *
                        p.d_chunks.d + c;
        }
#pragma unroll
        for (int j = 0; j < kAppUnroll; ++j) {
            if (!live[j]) continue;
            kc[to[j]] = x[j];
            vc[to[j]] = y[j];
        }
    }
}

int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

}  // namespace

cudaError_t launch_paged_tables(const TablesArgs &a, cudaStream_t st) {
    TablesParams p{a, log2_of(a.page_size), device_status_ptr()};
    auto smem = [](size_t requests) { return (3 * requests + 1) * sizeof(int); };
    // Threads for the rows, and for the requests and the pages they can get,
    // but no more than two blocks an SM: each forms the sums, which is most of
    // what it issues (1024 prompts, 528 thousand rows: one block an SM 10.9
    // us, two 8.3, four 10.9).
    constexpr int kBlocks = 2 * kSms;
    const int per_thread = a.total > kBlocks * kTabThreads ? 4 : 1;
    const long long items = std::max((a.total + per_thread - 1ll) / per_thread, a.B + (long long)a.total / a.page_size);
    const unsigned grid = (unsigned)std::min((items + kTabThreads - 1) / kTabThreads, (long long)kBlocks);
    return launch_after(per_thread == 4 ? paged_tables_kernel<4> : paged_tables_kernel<1>, grid, kTabThreads,
                        DynSmem(smem(a.B), smem(FA_PAGED_TABLES_MAX_B)), st, p);
}

cudaError_t launch_paged_append(const AppendArgs &a, cudaStream_t st) {
    AppendParams p;
    p.a = a;
    p.d_chunks = fast_div(a.d / 8);
    p.chunks = fast_div(a.Hkv * (a.d / 8));
    p.rows_per_block = p.chunks.d >= 1024 ? 1 : 1024 / p.chunks.d;
    p.shift = log2_of(a.page_size);
    p.status = device_status_ptr();
    const unsigned blocks = (unsigned)((a.total + (long long)p.rows_per_block - 1) / p.rows_per_block);
    return launch_after(paged_append_kernel, blocks, kAppThreads, 0, st, p);
}

}  // namespace fa
