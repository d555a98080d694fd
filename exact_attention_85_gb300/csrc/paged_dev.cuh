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

// Whether a request may have rows from .. to - 1.
__device__ __forceinline__ bool sound_rows(const PagedArgs &a, int from, int to) {
    return from >= 0 && to >= from && to <= a.total && to - from <= a.max_new;
}

// False if what the device holds for request b breaks the rules of the call
// (offsets, row bound, length): it then has no rows.
__device__ __forceinline__ bool load_request(const PagedArgs &a, int b, Request &r) {
    r.row0 = b;
    r.n = 1;
    if (a.cu_seqlens) {
        r.row0 = a.cu_seqlens[b];
        const int end = a.cu_seqlens[b + 1];
        if (!sound_rows(a, r.row0, end)) return false;
        r.n = end - r.row0;
    }
    r.len = a.seq_lens[b];
    return r.len >= 0 && r.len <= (a.max_pages << a.shift);
}

__host__ __device__ __forceinline__ int operator/(int x, const FastDiv &f) {
#ifdef __CUDA_ARCH__
    return (int)((__umulhi((uint32_t)x, f.mul) + (uint32_t)x) >> f.shift);
#else
    return x / f.d;
#endif
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long x) {
#pragma unroll
    for (int s = 16; s; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
    return x;
}

// Sum of the lanes' counts, each below 2^48 and all of them below 2^56: in
// two halves, as there is no 64-bit reduction.
__device__ __forceinline__ long long warp_count(long long x) {
    const unsigned lo = __reduce_add_sync(0xffffffffu, (unsigned)x & 0xFFFFFFu);
    const unsigned hi = __reduce_add_sync(0xffffffffu, (unsigned)(x >> 24));
    return ((long long)hi << 24) + lo;
}

// [u0, u1): the units of CTA c of G that share T units, and the CTA that has
// unit u.  The first T % G CTAs take one more than the others.
struct Ranges {
    long long each, more;
    __device__ __forceinline__ Ranges(long long T, int G) : each(T / G), more(T % G) {}
    __device__ __forceinline__ long long start(int c) const { return c * each + min((long long)c, more); }
    __device__ __forceinline__ int owner(long long u) const {
        const long long big = more * (each + 1);
        return (int)(u < big ? u / (each + 1) : more + (u - big) / each);
    }
};

// Weights are formed as 2^(score - maximum + this), log2 units, and so are
// their sums.  fp16 has no more than 2^-24 below 1, and a maximum lags by up
// to 2^8: keys 25 units below a row's largest would drop out, and those 14
// below lose bits, which shows where there are many of them (one key 17.6 in
// the natural log above 2^17 others, which have 0.3 % of the weight together:
// none of it was left).  At 2^15 of 2^16 fp16 has seven units more; scores of
// 10^7 and above, which are off by whole units themselves, can pass that and
// are held to fp16's largest number.
template <bool BF16>
constexpr float kWeightUnits = BF16 ? 0.0f : 7.0f;

// ------------------------------------------------- units of the two kernels

// Keys per tile of the few-row kernel (32 KB of K and V).
template <int D>
constexpr int kFewKeys = D == 128 ? 64 : 128;

// First tile and number of tiles of a (request, key/value head) pair; at
// least one, so that rows that see nothing are written.
template <int TK>
__device__ __forceinline__ int pair_tiles(const PagedArgs &a, const Request &r, int &t0) {
    const int lo = a.window > 0 ? max(0, r.len - r.n + 1 - a.window) : 0;
    t0 = lo / TK;
    return max(1, (r.len + TK - 1) / TK - t0);
}

// Work of the 256-row kernel, in key tiles.  A row block costs its tiles and
// as much as three more for the change from the block before (first Q, K and
// S with nothing to overlap, last P V and epilogue).  Counted among the units,
// so that CTAs whose range has many short blocks get fewer tiles.  Where there
// are only a few tiles for every SM it would only keep SMs idle.
constexpr int kBlockCost = 3;
struct WideWork {
    long long tiles, blocks;
    __device__ __forceinline__ int block_cost() const { return tiles > 4 * kSms ? kBlockCost : 0; }
    __device__ __forceinline__ long long units() const { return tiles + blocks * block_cost(); }
};

// Key tiles of a range; at least one.
__host__ __device__ __forceinline__ int range_tiles(int lo, int hi) {
    return max(1, (hi + kWideKeys - 1) / kWideKeys - lo / kWideKeys);
}

// Row blocks of a request in the 256-row kernel, and its own keys that block
// k of it sees.
__host__ __device__ __forceinline__ int blocks_of(const Request &r, const FastDiv &group) {
    return (int)(((unsigned)(r.n * group.d) + kWideRows - 1) / kWideRows);
}
__host__ __device__ __forceinline__ void block_keys(const PagedArgs &a, const FastDiv &group, const Request &r, int k,
                                                    int &lo, int &hi) {
    const int first = (k * kWideRows) / group;
    const int last =
        (r.n * group.d - k * kWideRows > kWideRows ? (k + 1) * kWideRows - 1 : r.n * group.d - 1) / group;
    hi = max(0, r.len - r.n + last + 1);
    // places below it, by the first row; in a tree any may hang on the context
    const int seen = r.len - r.n + (a.parents ? 0 : first) + 1;
    lo = a.window > 0 && seen > a.window ? seen - a.window : 0;
}
// First place that a row which sees places below hi sees under a window; what
// would pass 32 bits is below every place.
__host__ __device__ __forceinline__ int window_low(int hi, int window) {
    return max(hi, window - 0x7FFFFFFF) - window;
}
// Key tiles of the shared prefix that block k sees where they are read with
// its own, and the first key of them.
__host__ __device__ __forceinline__ int block_front(const PagedArgs &a, const FastDiv &group, const Request &r, int k,
                                                    int &lo) {
    lo = 0;
    if (a.window > 0) {
        const long long at = (long long)a.prefix_len + r.len - r.n + (k * kWideRows) / group + 1 - a.window;
        lo = (int)max(0ll, min(at, (long long)a.prefix_len));
    }
    return lo < a.prefix_len ? range_tiles(lo, a.prefix_len) : 0;
}
// Key tiles of blocks from, from + step, .. below nb of a request, for one
// key/value head, and the most that one has.  A block's fit 32 bits, but all
// of a prompt of N tokens are N^2 g / 65536: past 2^31 at 4 million tokens of
// 8 grouped heads.
template <bool JOINED>
__host__ __device__ __forceinline__ long long blocks_tiles(const PagedArgs &a, const FastDiv &group, const Request &r,
                                                           int from, int nb, int step, int &longest) {
    long long sum = 0;
#pragma unroll 1  // 8 chunks of 512 on a prefix of 2k: 148.6 us, unrolled 151.6
    for (int k = from; k < nb; k += step) {
        int lo, hi, front_lo;
        block_keys(a, group, r, k, lo, hi);
        const int tiles = range_tiles(lo, hi) + (JOINED ? block_front(a, group, r, k, front_lo) : 0);
        sum += tiles;
        longest = max(longest, tiles);
    }
    return sum;
}

// Rows of q that requests have: [first_row, end_row).  Where the first or the
// last request's offsets break the rules (it is reported, and has no rows),
// the sound ones may have rows anywhere.
__device__ __forceinline__ int first_row(const PagedArgs &a) {
    if (!a.cu_seqlens) return 0;
    const int from = a.cu_seqlens[0];
    return sound_rows(a, from, a.cu_seqlens[1]) ? from : 0;
}
__device__ __forceinline__ int end_row(const PagedArgs &a) {
    if (!a.cu_seqlens) return a.B;
    const int to = a.cu_seqlens[a.B];
    return sound_rows(a, a.cu_seqlens[a.B - 1], to) ? to : a.total;
}
// First key of the prefix that request r's rows see (prefix_len: none).
__device__ __forceinline__ int prefix_low(const PagedArgs &a, const Request &r) {
    const long long lo = (long long)a.prefix_len + r.len - r.n + 1 - a.window;
    return a.window > 0 ? (int)max(0ll, min(lo, (long long)a.prefix_len)) : 0;
}
__device__ __forceinline__ WideWork prefix_work(const PagedArgs &a, int rows, int group, int lo) {
    const long long blocks = ((long long)rows * group + kWideRows - 1) / kWideRows * a.Hkv;
    return {blocks * range_tiles(lo, a.prefix_len), blocks};
}

// What every warp of a block adds up of the batch before the block's first
// barrier; its producer then takes the sums of all.
struct PlanSum {
    unsigned long long tiles, beside;  // of this kernel; of the one that runs beside it
    int blocks, low;                   // row blocks or pairs; first key of the prefix that a row sees
    int beside_blocks, longest;        // longest: tiles of a row block, at most
    unsigned long long light;          // 256-row kernel, trees: tiles of blocks of up to 128 rows
};

// Key tiles of a request's row blocks, each counted as if it saw all keys that
// any of them sees: what the few-row kernel knows of the 256-row one's work.
__device__ __forceinline__ long long block_tiles(const PagedArgs &a, const Request &r, int group, int &blocks) {
    blocks = (int)(((unsigned)(r.n * group) + kWideRows - 1) / kWideRows);
    return (long long)blocks * range_tiles(a.window > 0 ? max(0, max(0, r.len - r.n + 1) - a.window) : 0, r.len);
}

// The 256-row kernel is bound by the tensor cores and the few-row kernel by
// memory, so a shared prefix' pass, or the long chunks of a mixed batch, run
// beside the few-row kernel, each on SMs of its own: the number that the
// 256-row kernel gets.  Times in us, as measured: a unit of the 256-row
// kernel takes 2.05 on one SM, with 14 to start and end; a few-row pair 0.35
// and 0.5 a tile on one SM, but at least 1.6, with 6 to start; and both
// together 4.7 ns for each 32 KB, of which a few-row tile is one and a unit of
// the other kernel two.  That is 7.0 TB/s, the rate at which the few-row kernel
// alone reads the cache, charged to the 256-row kernel's tiles as well, most
// of which come from L2: it fits the times, but what the limit is has not been
// measured.  Where it is what counts, the 256-row kernel gets all SMs that
// cost the other nothing.  (256 requests of
// 64-2048 keys on a 16k prefix: 220 us with 48 SMs, 211 with 50, 205 with 58,
// 202 with 62, 211 with 70, 216 with 76; one after the other 272.)  32
// candidates, one a lane; each kernel decides for itself, so a difference
// would cost time only.
__device__ __forceinline__ int wide_sms(long long wide_units, long long few_tiles, long long few_pairs) {
    const int lane = threadIdx.x & 31, g = kSms * (32 - lane) / 33;
    const float units = (float)wide_units, tiles = (float)few_tiles, pairs = (float)few_pairs;
    const float wide = 14.f + units * 2.05f / (float)g;
    const float few = 6.f + fmaxf(0.0047f * (tiles + 2.f * units),
                                  fmaxf(0.5f * tiles + 0.35f * pairs, 1.6f * pairs) / (float)(kSms - g));
    // the least of the larger times, and the first to have it
    const uint32_t cost = __float_as_uint(fmaxf(wide, few)) & ~31u;
    const uint32_t best = __reduce_min_sync(0xffffffffu, cost | lane);
    return __shfl_sync(0xffffffffu, g, best & 31);
}

// Programmatic dependent launch: lets the stream's next kernel start as soon
// as every CTA of this one has started, and waits until the kernel before
// this one has finished and its writes are visible.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace fa
