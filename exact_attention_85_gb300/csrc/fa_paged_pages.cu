// fa_paged_pages.cu -- branching requests of a paged key/value cache: table
// rows that continue another one's (fa_paged_fork), copies of pages
// (fa_paged_copy), tokens moved together (fa_paged_compact) and pages given
// back (fa_paged_free).
#include "../../include/fa.h"
#include "host_util.h"
#include "mma_sync.cuh"
#include "paged.h"
#include "paged_dev.cuh"
#include "ptx.cuh"
#include "status.cuh"

#include <algorithm>

namespace fa {

namespace {

__device__ __forceinline__ int pages_of(int tokens, int shift) {
    return (int)(((unsigned)tokens + (1u << shift) - 1) >> shift);
}

// Exclusive sums of two counts a thread over the block's threads, and both
// totals; `sm`: two values a warp.
template <int THREADS>
__device__ __forceinline__ void block_sums(long long &a, long long &b, long long &a_all, long long &b_all,
                                           long long (*sm)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long a_in = a, b_in = b;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, a_in, s), y = __shfl_up_sync(0xffffffffu, b_in, s);
        if (lane >= s) {
            a_in += x;
            b_in += y;
        }
    }
    if (lane == 31) {
        sm[warp][0] = a_in;
        sm[warp][1] = b_in;
    }
    __syncthreads();
    a = a_in - a;
    b = b_in - b;
    a_all = b_all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) {
            a += sm[w][0];
            b += sm[w][1];
        }
        a_all += sm[w][0];
        b_all += sm[w][1];
    }
}

// The last of n entries (the first is 0) that is at most x.
__device__ __forceinline__ int last_at_most(const int *at, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (at[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// -------------------------------------------------------------------- fork

constexpr int kForkThreads = 256;
constexpr int kForkCells = 128;  // table cells of a warp's unit of work

struct ForkParams {
    ForkArgs a;
    int shift;  // log2(page_size)
    unsigned int *status;
};

// As in paged_tables_kernel every block forms the sums over all forks (pages
// needed, units of table cells) for itself, and then writes its share.  A unit
// is up to 128 cells of one fork, dealt over the grid's warps.  The holders of
// a page are counted once for all forks of a row: the first fork of the row
// that is served adds their number.  Bound by latency (lengths, cells, counts
// one behind the other) and, beside it, the calling program: 8 forks of 31
// pages 3.3 us, 960 forks of 500 thousand cells 7.2.
__global__ void __launch_bounds__(kForkThreads) paged_fork_kernel(const ForkParams p) {
    extern __shared__ int smem[];
    const int F = p.a.F;
    int *row = smem;          // [F] source row; -1: not served, -2: unsound
    int *len = row + F;       // [F]
    int *unit = len + F;      // [F] first unit
    int *fresh = unit + F;    // [F] new pages of the forks before
    __shared__ long long sm[kForkThreads / 32][2];
    const int tid = threadIdx.x, lane = tid & 31;
    const int per = (F + kForkThreads - 1) / kForkThreads | 1;  // odd: neighbouring threads in different banks
    const int f0 = min(F, tid * per), f1 = min(F, f0 + per);
    const int in_page = (1 << p.shift) - 1;
    wait_previous();
    launch_dependents();
    const int start_in = p.a.free_start ? *p.a.free_start : 0;
    const bool start_ok = start_in >= 0 && start_in <= p.a.num_free;
    const int start = start_ok ? start_in : 0, room = start_ok ? p.a.num_free - start : 0;
    bool bad = !start_ok;
#pragma unroll 4
    for (int f = tid; f < F; f += kForkThreads) {
        const int s = p.a.src[f], t = p.a.dst[f];
        const bool sound = s >= 0 && s < p.a.B && t >= 0 && t < p.a.B && s != t;
        const int n = sound ? p.a.seq_lens[s] : -1;
        const bool fits = n >= 0 && n <= (p.a.max_pages << p.shift);
        if (!fits) bad = true;
        row[f] = fits ? s : -2;
        len[f] = fits ? n : 0;
    }
    __syncthreads();
    auto units_of = [&](int n) { return ((n >> p.shift) + kForkCells - 1) / kForkCells; };
    long long need = 0, units = 0, n_all, u_all;
    for (int f = f0; f < f1; ++f) {
        need += (len[f] & in_page) != 0;
        units += units_of(len[f]);
    }
    block_sums<kForkThreads>(need, units, n_all, u_all, sm);
    for (int f = f0; f < f1; ++f) {
        const int nd = (len[f] & in_page) != 0;
        fresh[f] = (int)need;
        unit[f] = (int)min(units, 0x7FFFFFFFll);
        units += units_of(len[f]);
        need += nd;
        if (nd && need > room) row[f] = -1;
    }
    __syncthreads();
    if (bad && blockIdx.x == 0) record_bad_args(p.status);
    if (blockIdx.x == 0 && tid == 0) {
        p.a.counts[0] = start + (int)min(n_all, (long long)room);
        p.a.counts[1] = (int)max(n_all - room, 0ll);
    }
    const long long id = (long long)blockIdx.x * kForkThreads + tid, threads = (long long)gridDim.x * kForkThreads;
    for (long long f = id; f < F; f += threads) {
        const int n = len[f], s = row[f], t = p.a.dst[f], full = n >> p.shift;
        int from = -1, to = -1, rows = 0;
        if (s >= 0 && (n & in_page)) {
            from = p.a.block_table[(size_t)s * p.a.max_pages + full];
            to = p.a.free_pages[start + fresh[f]];
            rows = n & in_page;
            p.a.block_table[(size_t)t * p.a.max_pages + full] = to;
            if ((unsigned)from >= (unsigned)p.a.num_pages || (unsigned)to >= (unsigned)p.a.num_pages) {
                record_bad_args(p.status);
                from = to = -1;
                rows = 0;
            }
        }
        p.a.copies[f] = from;
        p.a.copies[F + f] = to;
        p.a.copies[2ll * F + f] = rows;
        if (s != -2) p.a.seq_lens[t] = s >= 0 ? n : 0;
    }
    const long long warps = threads / 32;
    const int all = (int)min(u_all, 0x7FFFFFFFll);
    for (long long u = id / 32; u < all; u += warps) {
        const int f = last_at_most(unit, F, (int)u), s = row[f];
        if (s < 0) continue;
        const int full = len[f] >> p.shift, c0 = ((int)u - unit[f]) * kForkCells;
        const int *from = p.a.block_table + (size_t)s * p.a.max_pages;
        int *to = p.a.block_table + (size_t)p.a.dst[f] * p.a.max_pages;
        int cell[kForkCells / 32];
#pragma unroll
        for (int i = 0; i < kForkCells / 32; ++i) {
            const int c = c0 + i * 32 + lane;
            cell[i] = c < full ? from[c] : -1;
        }
        // served forks of the row: none before this one?  how many behind it?
        int holders = 1;
        for (int g = 0; g < f && holders; g += 32)
            if (__any_sync(0xffffffffu, g + lane < f && row[g + lane] == s)) holders = 0;
        for (int g = f + 1; g < F && holders; g += 32)
            holders += __popc(__ballot_sync(0xffffffffu, g + lane < F && row[g + lane] == s));
#pragma unroll
        for (int i = 0; i < kForkCells / 32; ++i) {
            const int c = c0 + i * 32 + lane;
            if (c >= full) continue;
            to[c] = cell[i];
            if (!holders) continue;
            if ((unsigned)cell[i] < (unsigned)p.a.num_pages)
                atomicAdd(p.a.shares + cell[i], holders);
            else
                record_bad_args(p.status);
        }
    }
}

// -------------------------------------------------------------------- copy

constexpr int kCopyThreads = 256, kCopyUnroll = 4;

struct CopyParams {
    CopyArgs a;
    FastDiv pieces;  // blocks of a pair of pages
    int shift, head_shift;  // log2 of page_size, and of the 16-byte pieces of a head's rows of a page
    unsigned int *status;
};

// A block copies up to 16 KB of K and of V: the rows of some heads of a page,
// or a part of one head's, which lie one behind the other on both sides.  Bound
// by memory: 1.01 GB in and out in 150 us, 6.7 TB/s, the rate of a plain copy;
// 960 pages of 16 rows, 8 heads, 8 us.
__global__ void __launch_bounds__(kCopyThreads) paged_copy_kernel(const CopyParams p) {
    const int i = blockIdx.x / p.pieces, piece = blockIdx.x - i * p.pieces.d;
    wait_previous();
    launch_dependents();
    const int from = p.a.src[i], to = p.a.dst[i], rows = p.a.rows ? p.a.rows[i] : 1 << p.shift;
    if (from < 0 || to < 0) return;
    if (from >= p.a.num_pages || to >= p.a.num_pages || rows < 0 || rows > (1 << p.shift)) {
        record_bad_args(p.status);
        return;
    }
    const size_t at = (size_t)from * p.a.Hkv << p.head_shift, out = (size_t)to * p.a.Hkv << p.head_shift;
    const uint4 *k = static_cast<const uint4 *>(p.a.k_cache) + at, *v = static_cast<const uint4 *>(p.a.v_cache) + at;
    uint4 *ko = static_cast<uint4 *>(p.a.k_cache) + out, *vo = static_cast<uint4 *>(p.a.v_cache) + out;
    const int all = p.a.Hkv << p.head_shift, mask = (1 << p.head_shift) - 1;
    const int c0 = piece * (kCopyThreads * kCopyUnroll) + threadIdx.x, end = rows << (p.head_shift - p.shift);
    uint4 x[kCopyUnroll], y[kCopyUnroll];
#pragma unroll
    for (int j = 0; j < kCopyUnroll; ++j) {
        const int c = c0 + j * kCopyThreads;
        if (c >= all || (c & mask) >= end) continue;
        x[j] = __ldcs(k + c);
        y[j] = __ldcs(v + c);
    }
#pragma unroll
    for (int j = 0; j < kCopyUnroll; ++j) {
        const int c = c0 + j * kCopyThreads;
        if (c >= all || (c & mask) >= end) continue;
        ko[c] = x[j];
        vo[c] = y[j];
    }
}

// ----------------------------------------------------------------- compact

constexpr int kMoveThreads = 256, kMoveUnroll = 4;
constexpr int kMoveBytes = kMoveThreads * kMoveUnroll * 16;  // of a tile of rows
constexpr int kMoveStages = 3;                               // tiles in shared memory
constexpr int kMoveLook = kMoveUnroll / 2;                   // rows of a tile that a thread looks up, at most
constexpr int kMoveSlots = kMoveStages + 1;                  // tiles whose slots are known

constexpr unsigned kStays = 0xFFFFFFFFu;

struct CompactParams {
    CompactArgs a;
    FastDiv heads;         // 2 Hkv: K's and V's planes of a page
    int shift, row_bytes;  // log2(page_size); 2 d
    int split, cols;       // blocks of a row; 16-byte pieces of a row that one has
    unsigned int *status;
};

// In place: token base + i gets token base + keep[i], keep[i] >= i, increasing.
// A block takes some columns of one head of a request, K or V, and walks the
// kept tokens tile by tile, with the loads of two tiles ahead of the stores.
// What a later tile reads lies behind everything that this one and those
// before it write (keep[j] >= j), so it may be read early; a tile's own reads
// have landed, in every thread, before its first write.  Blocks never touch
// one another's bytes.  Bound by the memory's bandwidth at short pieces: 302 MB
// in and out in 57 us, 5.3 TB/s.  (A copy is on its way for one to two tiles;
// 128 threads with twice the pieces each took 67 us, slots that are looked up
// when they are needed 106, as a tile then takes two loads' latency.)
__global__ void __launch_bounds__(kMoveThreads) paged_compact_kernel(const CompactParams p) {
    extern __shared__ __align__(16) uint8_t move_smem[];  // [kMoveStages] tiles, then slots
    const int tid = threadIdx.x;
    int unit = blockIdx.x / p.split;
    const int col0 = (blockIdx.x - unit * p.split) * p.cols;
    const int b = unit / p.heads, plane = unit - b * p.heads.d;  // K's heads, then V's
    const int h = plane >= p.a.Hkv ? plane - p.a.Hkv : plane;
    const int rows = kMoveThreads * kMoveUnroll / p.cols;  // of a tile
    // [kMoveSlots][rows]: from and to, rows of the cache's heads (kStays: none)
    uint2 *slots = reinterpret_cast<uint2 *>(move_smem + kMoveStages * kMoveBytes);
    wait_previous();
    launch_dependents();
    const int n = p.a.keep_lens[b], base = p.a.base_lens[b];
    const int room = p.a.max_pages << p.shift;
    if (n < 0 || n > p.a.max_keep || base < 0 || base > room || n > room - base) {
        if (plane == 0 && tid == 0) record_bad_args(p.status);
        return;
    }
    const int *keep = p.a.keep + (size_t)b * p.a.max_keep, *table = p.a.block_table + (size_t)b * p.a.max_pages;
    uint8_t *cache = static_cast<uint8_t *>(plane >= p.a.Hkv ? p.a.v_cache : p.a.k_cache) + col0 * 16;
    const int tiles = (n + rows - 1) / rows;
    // Looking up a row's slots takes two loads, one behind the other: its kept
    // token, and the pages of both places.  Each is started a tile before its
    // result is needed.
    int k[kMoveLook], prev[kMoveLook], from[kMoveLook], page_from[kMoveLook], page_to[kMoveLook];
    const int mask = (1 << p.shift) - 1;
    auto fetch_keep = [&](int t) {
#pragma unroll
        for (int q = 0; q < kMoveLook; ++q) {
            const int r = tid + q * kMoveThreads, i = t * rows + r;
            k[q] = i;  // stays
            prev[q] = -1;
            if (t >= tiles || r >= rows || i >= n) continue;
            k[q] = keep[i];
            if (i) prev[q] = keep[i - 1];
        }
    };
    auto fetch_pages = [&](int t) {
#pragma unroll
        for (int q = 0; q < kMoveLook; ++q) {
            const int i = t * rows + tid + q * kMoveThreads;
            from[q] = -1;
            if (k[q] == i && prev[q] < i) continue;
            if (k[q] <= prev[q] || k[q] < i || k[q] >= room - base) {
                record_bad_args(p.status);
                continue;
            }
            from[q] = base + k[q];
            page_from[q] = table[from[q] >> p.shift];
            page_to[q] = table[(base + i) >> p.shift];
        }
    };
    auto put_slots = [&](int t) {
#pragma unroll
        for (int q = 0; q < kMoveLook; ++q) {
            const int r = tid + q * kMoveThreads, i = t * rows + r;
            if (t >= tiles || r >= rows) continue;
            uint2 s = make_uint2(kStays, kStays);
            if (from[q] >= 0) {
                if ((unsigned)page_from[q] < (unsigned)p.a.num_pages && (unsigned)page_to[q] < (unsigned)p.a.num_pages)
                    s = make_uint2((((unsigned)page_from[q] * p.a.Hkv + h) << p.shift) + (from[q] & mask),
                                   (((unsigned)page_to[q] * p.a.Hkv + h) << p.shift) + ((base + i) & mask));
                else
                    record_bad_args(p.status);
            }
            slots[t % kMoveSlots * rows + r] = s;
        }
    };
    const int row = tid / p.cols, step = kMoveThreads / p.cols;
    uint8_t *const column = cache + (tid - row * p.cols) * 16;
    auto at = [&](unsigned r) { return reinterpret_cast<uint4 *>(column + (size_t)r * p.row_bytes); };
    const uint32_t mine = smem_u32(move_smem) + tid * 16;  // a thread's pieces are its own
    auto load = [&](int t) {
        if (t < tiles) {
            const uint2 *s = slots + t % kMoveSlots * rows + row;
            const uint32_t to = mine + t % kMoveStages * kMoveBytes;
            unsigned r[kMoveUnroll];
#pragma unroll
            for (int j = 0; j < kMoveUnroll; ++j) r[j] = s[j * step].x;
#pragma unroll
            for (int j = 0; j < kMoveUnroll; ++j)
                if (r[j] != kStays) cp_async_16(to + j * kMoveThreads * 16, at(r[j]));
        }
        cp_async_commit();
    };
    // lines of keep[], a tile's by its threads, eight tiles ahead: from memory
    // they would take longer than a tile
    auto prefetch_keep = [&](long long i) {
        if (i < n) asm volatile("prefetch.global.L2 [%0];" ::"l"(keep + i));
    };
    for (int i = tid * 32; i < 8 * rows; i += 32 * kMoveThreads) prefetch_keep(i);
    for (int t = 0; t < kMoveStages - 1; ++t) {
        fetch_keep(t);
        fetch_pages(t);
        put_slots(t);
    }
    __syncthreads();
    for (int t = 0; t < kMoveStages - 1; ++t) load(t);
    fetch_keep(kMoveStages - 1);
    fetch_pages(kMoveStages - 1);
    fetch_keep(kMoveStages);
    for (int t = 0; t < tiles; ++t) {
        put_slots(t + kMoveStages - 1);
        fetch_pages(t + kMoveStages);
        fetch_keep(t + kMoveStages + 1);
        if (tid * 32 < rows) prefetch_keep((t + 8ll) * rows + tid * 32);
        cp_async_wait<kMoveStages - 2>();
        __syncthreads();
        load(t + kMoveStages - 1);
        const uint2 *s = slots + t % kMoveSlots * rows + row;
        const uint4 *x = reinterpret_cast<const uint4 *>(move_smem + t % kMoveStages * kMoveBytes) + tid;
        unsigned r[kMoveUnroll];
        uint4 y[kMoveUnroll];
#pragma unroll
        for (int j = 0; j < kMoveUnroll; ++j) {
            r[j] = s[j * step].y;
            y[j] = x[j * kMoveThreads];
        }
#pragma unroll
        for (int j = 0; j < kMoveUnroll; ++j)
            if (r[j] != kStays) *at(r[j]) = y[j];
    }
}

// -------------------------------------------------------------------- free

constexpr int kFreeThreads = 1024, kFreeWarps = kFreeThreads / 32;
constexpr int kFreeCtas = 16;  // of the one cluster, at most
constexpr int kFreeKept = 16;  // cells whose pages a lane keeps
// What stands in shares[] for a page that falls free, while the call runs:
// below every count, the lower the earlier the first cell that gives it up.
constexpr int kFreeCode = -(1 << 30);

struct FreeParams {
    FreeArgs a;
    int shift;
    unsigned int *status;
};

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int cluster_load(const int *mine, int rank) {
    uint32_t at;
    int x;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(at)
                 : "r"((uint32_t)__cvta_generic_to_shared(mine)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
    return x;
}

// All given-up cells are numbered in order of (request, cell); a warp has an
// equal, contiguous range of them.  With shared pages:
//   1  every cell takes one from its page's count: below 0, the page is free
//   2  every cell of a free page writes its number there, the lowest stays
//   3  the cell that finds its own number has the page; they are counted
//   4  and write the pages, by the counts of the warps before, and the zeros
// with barriers of the cluster between them.  Without, every cell has its page.
// Bound by scattered accesses, four a cell, of at most 16 SMs: one launch with
// one cluster is what this takes for its barriers, at the price of the GPU's
// other SMs.  131 thousand cells of 1024 requests 35 us, without counts 16 (with
// 8 CTAs that looked the pages up in every pass 87); 30 cells of 16 requests
// 7.3, most of it start and sums.
template <bool SHARED>
__global__ void __launch_bounds__(kFreeThreads) paged_free_kernel(const FreeParams p) {
    extern __shared__ int smem[];
    const int B = p.a.B;
    int *first = smem;      // [B] number of a request's first cell
    int *col = smem + B;    // [B] its column
    __shared__ long long sm[kFreeWarps][2];
    __shared__ int warp_freed[kFreeWarps], cta_freed;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (B + kFreeThreads - 1) / kFreeThreads | 1;
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    const int rank = blockIdx.x, ctas = gridDim.x;
    wait_previous();
    launch_dependents();
    const int start_in = *p.a.free_start;
    const bool start_ok = start_in >= 0 && start_in <= p.a.num_free;
    const int start = start_ok ? start_in : 0;
    bool bad = !start_ok;
    for (int b = tid; b < B; b += kFreeThreads) {
        const int o = p.a.old_lens[b], n = p.a.new_lens[b];
        const bool sound = n >= 0 && n <= o && o <= (p.a.max_pages << p.shift);
        if (!sound) bad = true;
        col[b] = sound ? pages_of(n, p.shift) : 0;
        first[b] = sound ? pages_of(o, p.shift) - col[b] : 0;
    }
    __syncthreads();
    long long cells = 0, none = 0, all, none_all;
    for (int b = b0; b < b1; ++b) cells += first[b];
    block_sums<kFreeThreads>(cells, none, all, none_all, sm);
    for (int b = b0; b < b1; ++b) {
        const int n = first[b];
        first[b] = (int)cells;
        cells += n;
    }
    __syncthreads();
    if (bad && rank == 0) record_bad_args(p.status);
    const int E = (int)all;  // at most 2^30: the entry point sees to it
    const int units = (E + 31) / 32, each = (units + ctas * kFreeWarps - 1) / (ctas * kFreeWarps);
    const int u0 = min(units, (rank * kFreeWarps + warp) * each), u1 = min(units, u0 + each);  // of 32 cells
    // the page of cell e, -1 if there is none, or none of that number
    auto page_of = [&](int e) {
        if (e >= E) return -1;
        const int b = last_at_most(first, B, e);
        const int page = p.a.block_table[(size_t)b * p.a.max_pages + col[b] + e - first[b]];
        if ((unsigned)page < (unsigned)p.a.num_pages) return page;
        record_bad_args(p.status);
        return -1;
    };
    // A lane keeps the pages of its first cells, which are all of them but for
    // very long tables, and looks the others up in every pass again.
    int kept[kFreeKept];
#pragma unroll
    for (int i = 0; i < kFreeKept; ++i) kept[i] = u0 + i < u1 ? page_of((u0 + i) * 32 + lane) : -1;
    auto for_each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < kFreeKept; ++i)
            if (u0 + i < u1) f((u0 + i) * 32 + lane, kept[i], i);
#pragma unroll 1
        for (int u = u0 + kFreeKept; u < u1; ++u) f(u * 32 + lane, page_of(u * 32 + lane), kFreeKept);
    };
    int *shares = p.a.shares;
    if (SHARED) {
        unsigned seen_free = 0;  // of the kept cells, whose page fell free with them or before
        for_each([&](int, int page, int i) {
            if (page < 0) return;
            if (i == kFreeKept)
                atomicSub(shares + page, 1);
            else if (atomicSub(shares + page, 1) <= 0)
                seen_free |= 1u << i;
        });
        cluster_sync();
        for_each([&](int e, int page, int i) {
            if (page < 0) return;
            if ((i < kFreeKept && seen_free >> i & 1) || __ldcg(shares + page) < 0)
                atomicMin(shares + page, kFreeCode - (E - 1 - e));
        });
        cluster_sync();
    }
    unsigned has = 0;  // of the kept cells, which have their page
    int mine = 0;
    auto frees = [&](int e, int page) {
        return page >= 0 && (!SHARED || __ldcg(shares + page) == kFreeCode - (E - 1 - e));
    };
    for_each([&](int e, int page, int i) {
        const bool f = frees(e, page);
        if (f && i < kFreeKept) has |= 1u << i;
        mine += __popc(__ballot_sync(0xffffffffu, f));
    });
    if (lane == 0) warp_freed[warp] = mine;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kFreeWarps; ++w) {
        if (w < warp) before += warp_freed[w];
        total += warp_freed[w];
    }
    if (ctas > 1) {
        if (tid == 0) cta_freed = total;
        cluster_sync();
        // a CTA's number by each of the first lanes
        const int theirs = lane < ctas ? cluster_load(&cta_freed, lane) : 0;
        total = __reduce_add_sync(0xffffffffu, theirs);
        before += __reduce_add_sync(0xffffffffu, lane < rank ? theirs : 0);
        cluster_sync();  // no CTA leaves, and nobody clears a code, before all have read
    }
    int to = start - total + before;
    for_each([&](int e, int page, int i) {
        const bool f = i < kFreeKept ? has >> i & 1 : frees(e, page);
        const unsigned who = __ballot_sync(0xffffffffu, f);
        if (f) {
            const int k = to + __popc(who & ((1u << lane) - 1));
            if (k >= 0) p.a.free_pages[k] = page;
            if (SHARED) shares[page] = 0;
        }
        to += __popc(who);
    });
    if (rank == 0 && tid == 0) {
        p.a.counts[0] = max(0, start - total);
        p.a.counts[1] = max(0, total - start);
        if (total > start) record_bad_args(p.status);
    }
}

int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

}  // namespace

cudaError_t launch_paged_fork(const ForkArgs &a, cudaStream_t st) {
    ForkParams p{a, log2_of(a.page_size), device_status_ptr()};
    auto smem = [](size_t forks) { return 4 * forks * sizeof(int); };
    // a warp for each unit of cells that there can be, two blocks an SM at most
    const long long units = (long long)a.F * ((a.max_pages + kForkCells - 1) / kForkCells);
    const unsigned grid = (unsigned)std::min((units + kForkThreads / 32 - 1) / (kForkThreads / 32), 2ll * kSms);
    return launch_after(paged_fork_kernel, grid, kForkThreads, DynSmem(smem(a.F), smem(FA_PAGED_FORK_MAX)), st, p);
}

// Blocks of a pair of pages.
static long long copy_pieces(int Hkv, int d, int page_size) {
    constexpr int kBlock = kCopyThreads * kCopyUnroll;
    return ((long long)Hkv * page_size * (d / 8) + kBlock - 1) / kBlock;
}
long long copy_blocks(int n, int Hkv, int d, int page_size) { return n * copy_pieces(Hkv, d, page_size); }

cudaError_t launch_paged_copy(const CopyArgs &a, cudaStream_t st) {
    CopyParams p;
    p.a = a;
    p.shift = log2_of(a.page_size);
    p.head_shift = log2_of(a.page_size * (a.d / 8));
    p.pieces = fast_div((int)copy_pieces(a.Hkv, a.d, a.page_size));
    p.status = device_status_ptr();
    return launch_after(paged_copy_kernel, (unsigned)copy_blocks(a.n, a.Hkv, a.d, a.page_size), kCopyThreads, 0, st, p);
}

cudaError_t launch_paged_compact(const CompactArgs &a, cudaStream_t st) {
    CompactParams p;
    p.a = a;
    p.shift = log2_of(a.page_size);
    p.row_bytes = 2 * a.d;
    p.heads = fast_div(2 * a.Hkv);
    p.status = device_status_ptr();
    // Blocks of a row's columns, 32 bytes at least, until there is one an SM.
    // 128 units of 4096 .. 8191 rows of 256 bytes: 78 us with a block each, 57
    // with two, 65 with four, 72 with eight: short pieces of a row cost more
    // instructions and more of the memory's bandwidth than they fill.
    const long long units = 2ll * a.B * a.Hkv;
    p.split = 1;
    while (p.row_bytes / p.split > 32 && units * p.split < kSms) p.split *= 2;
    p.cols = p.row_bytes / p.split / 16;
    auto smem = [](int cols) {
        return (size_t)kMoveStages * kMoveBytes + kMoveSlots * (kMoveThreads * kMoveUnroll / cols) * sizeof(uint2);
    };
    return launch_after(paged_compact_kernel, (unsigned)(units * p.split), kMoveThreads,
                        DynSmem(smem(p.cols), smem(2)), st, p);
}

cudaError_t launch_paged_free(const FreeArgs &a, cudaStream_t st) {
    FreeParams p{a, log2_of(a.page_size), device_status_ptr()};
    auto smem = [](size_t requests) { return 2 * requests * sizeof(int); };
    // CTAs of 4 cells a thread, as many as there can be cells for
    unsigned grid = 1;
    while (grid < kFreeCtas && (long long)a.B * a.max_pages > (long long)grid * 4 * kFreeThreads) grid *= 2;
    auto kernel = a.shares ? paged_free_kernel<true> : paged_free_kernel<false>;
    if (grid > 8) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    return launch_cluster_after(kernel, grid, grid, kFreeThreads, DynSmem(smem(a.B), smem(FA_PAGED_TABLES_MAX_B)), st,
                                p);
}

}  // namespace fa
