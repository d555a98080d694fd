// fa_fwd_paged_wide.cu -- forward attention from a paged key/value cache for
// many query rows: prompts read in by chunks, and the rows of a whole batch
// against a prefix that all its requests share.
//
// A segment of work is 256 query rows of one key/value head and a range of
// its key tiles.  A row is a (token, query head) pair: the g = Hq / Hkv heads
// that read the key/value head are neighbouring rows of the tile, so grouped
// heads share every K/V tile that is read, and with a shared prefix so do all
// requests (their rows stand one behind the other in q).  The loop is that of
// the dense forward (fa_fwd.cu): two 128-row Q tiles A and B walk the same
// K/V stream, their softmax warpgroups take turns on the tensor cores, O is
// rescaled lazily and exactly, and P is read from tensor memory.  What
// differs: K/V tiles are gathered page by page (one TMA box per page and
// 64-column half), Q rows are copied into the swizzled operand layout by the
// helper warps, and every row has its own visible range of keys.
//
// The key tiles of all (row block, key/value head) pairs are numbered in
// order and every CTA (one per SM) takes an equal, contiguous range, as in
// the few-row kernel: chunks behind contexts of any lengths then keep all SMs
// busy to the end, at the price of merging the blocks that a range's border
// cuts (at most one border a CTA); where blocks are short, none is cut and a
// CTA takes those that begin in its range.  The K/V ring, the barriers and
// the tensor memory carry on from segment to segment; the next segment's Q is
// loaded and its first S issued before the epilogue of the one before.
//   warps 0-3 softmax + epilogue of tile A, 4-7 of tile B, 8 producer (plans
//   the segments and tells the others), 9 MMA issuer (owns the tensor memory),
//   10-11 helpers (Q, the V rows that nobody may see, and the paths of trees)
#include "../../include/fa.h"
#include "host_util.h"
#include "mma_sync.cuh"
#include "paged.h"
#include "paged_dev.cuh"
#include "ptx.cuh"

#include <type_traits>

namespace fa {

namespace {

constexpr int kBM = 128, kBN = 128;
constexpr int kRows = kWideRows;
static_assert(kRows == 2 * kBM && kBN == kWideKeys, "tile sizes of the plan");
constexpr int kThreads = 384;
constexpr int kHelperWarps = 2;
constexpr int kProducerWarp = 8, kMmaWarp = 9;
constexpr float kRescaleThreshold = 8.0f;
// Key tiles of a segment where the table may hold longer blocks (LONG).  The
// tensor cores cut every product to some 25 bits below the leading one of the
// sum before they add it, always towards less, so a sum of n terms loses up to
// n 2^-26 of itself: with 512 rows behind a million keys, values of mean 1, O
// was off by 4.9e-3, where storing fp16 makes 2.2e-4 and bf16 1.7e-3.  Sums of
// 2^15 keys (fp16) or 2^17 (bf16) lose a fraction of that; they are added up
// in fp32, in memory.  A kernel of its own, as the others would be 2 to 3 %
// slower for it (chunks 143.6 and 147 us).
template <bool BF16>
constexpr int kMaxTiles = BF16 ? 1024 : 256;
constexpr uint32_t kColS = 0, kColO = 256;  // + 128 per tile

// Requests whose tile counts the producer finds in shared memory (a multiple
// of 32), in 32 bits each: there is no room for 64.  It forms larger ones anew.
constexpr int kKept = 256;
constexpr unsigned kMany = 0xFFFFFFFFu;

template <int D>
struct WideLayout {
    static constexpr int KS = D == 128 ? 3 : 4;
    static constexpr int VS = D == 128 ? 2 : 4;
    static constexpr int NBOX = D / 64;
    static constexpr int TILE = 128 * D * 2;
    static constexpr int BOX = 128 * 128;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + 2 * TILE;
    static constexpr int OFF_V = OFF_K + KS * TILE;
    static constexpr int OFF_BAR = OFF_V + VS * TILE;
    // q_full, k_full[KS], k_empty[KS], v_full[VS], v_empty[VS], s_full[2],
    // p_full[2], o_final[2], seg_full[2], seg_empty[2], q_empty, v_clean[VS], drain,
    // tree_full[2]
    static constexpr int NBAR = 1 + 2 * KS + 3 * VS + 2 + 2 + 2 + 2 + 2 + 2 + 2;
    static constexpr int OFF_SEG = (OFF_BAR + NBAR * 8 + 15) & ~15;  // [2]
    static constexpr int OFF_MISC = OFF_SEG + 2 * 64;
    static constexpr int OFF_KEPT = OFF_MISC + 16 + kThreads / 32 * (int)sizeof(PlanSum);
    static constexpr int BYTES = OFF_KEPT + kKept * 4;
    static constexpr int ALLOC = BYTES + 1024;
    static_assert(ALLOC <= 227 * 1024, "shared memory");
};

struct WideParams {
    PagedArgs a;
    FastDiv group;  // query heads per key/value head
    int prefix;  // 1: rows of the whole batch against the shared prefix
    int shared;  // the few-row kernel runs at the same time
    int above;   // own pass: only requests of more rows a pair
    int q_box;   // tokens of a 128-row Q tile if the group divides it (TMA), else 0
    int after;   // runs beside the call's kernel before, which has waited for what came before
    int o32;     // O is 32-byte aligned (the entry points promise 16)
    PartView part;
    float scale_log2;
    unsigned int *status;
};

// Part of a row block's keys, as the producer tells it to the others.
struct Segment {
    int row0, n, len;    // rows of q and keys of the request (prefix: of the batch, of the prefix)
    int r0;              // first row of the block, counted in (token, head) pairs
    int hk, j0, nj;      // key/value head; first of the block's key tiles, number of them (-1: the end)
    int front, front_lo; // tiles of the shared prefix before its own; first key of those that some row sees
    int key_lo, key_hi;  // keys of its own (prefix pass: of the prefix) that some row sees
    int code;            // of the block's rows (PartView), 0 if the block is whole
    int slot;            // -1: whole, else the CTA's slot that the part goes to
    int more;            // kBefore, kBehind: this CTA has tiles of the block before these, and behind them
    int pad[2];
};
enum : int { kBefore = 1, kBehind = 2 };
static_assert(sizeof(Segment) == 64, "shared-memory slot");

// Key tile i of a segment: the prefix' tiles come first, where JOINED.
template <bool JOINED>
struct KeyTile {
    int kv0, lo, hi;  // first key; keys some row of the block sees
    bool in_front;
    __device__ __forceinline__ KeyTile(const Segment &sg, int i, int prefix_len) {
        const int j = sg.j0 + i;
        in_front = JOINED && j < sg.front;
        lo = in_front ? sg.front_lo : sg.key_lo;
        hi = in_front ? prefix_len : sg.key_hi;
        kv0 = (lo / kBN + j - (!JOINED || in_front ? 0 : sg.front)) * kBN;
    }
    // Whether it holds keys that no row of the block sees.
    __device__ __forceinline__ bool hides() const { return kv0 < lo || kv0 + kBN > hi; }
};

// The request of a row of q: the last one that starts at or before it.
__device__ __forceinline__ int request_of(const PagedArgs &a, int row) {
    if (!a.cu_seqlens) return row;
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.cu_seqlens[mid] <= row) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Keys that block k of a request sees: its own, or the prefix' in that pass.
__device__ __forceinline__ void block_keys(const WideParams &p, const Request &r, int k, int prefix_lo, int &lo,
                                           int &hi) {
    lo = prefix_lo;
    hi = r.len;
    if (!p.prefix) block_keys(p.a, p.group, r, k, lo, hi);
}
// Key tiles of the shared prefix that block k sees, and the first key of them.
template <bool JOINED>
__device__ __forceinline__ int block_front(const WideParams &p, const Request &r, int k, int &lo) {
    lo = 0;
    return JOINED ? block_front(p.a, p.group, r, k, lo) : 0;
}
// All key tiles of block k.
template <bool JOINED>
__device__ __forceinline__ int tiles_of(const WideParams &p, const Request &r, int k, int prefix_lo) {
    int lo, hi, front_lo;
    block_keys(p, r, k, prefix_lo, lo, hi);
    return block_front<JOINED>(p, r, k, front_lo) + range_tiles(lo, hi);
}
// Key tiles of all blocks of a request, for one key/value head, and the most
// that a block has.
struct RequestTiles {
    long long sum;
    int longest;
};
// The sums of 32 requests, one a lane: each lane walks its request's blocks,
// or the warp one request's after the other's, whichever takes fewer steps.
template <bool JOINED>
__device__ __noinline__ RequestTiles request_tiles(const WideParams &p, Request r, int nb, int lane) {
    RequestTiles t{0, 0};
    const unsigned some = __ballot_sync(0xffffffffu, nb > 0);
    if ((int)__reduce_max_sync(0xffffffffu, nb) <= __popc(some)) {
        t.sum = blocks_tiles<JOINED>(p.a, p.group, r, 0, nb, 1, t.longest);
        return t;
    }
    for (unsigned left = some; left; left &= left - 1) {
        const int i = __ffs(left) - 1, n = __shfl_sync(0xffffffffu, nb, i);
        Request o;
        o.row0 = 0;
        o.n = __shfl_sync(0xffffffffu, r.n, i);
        o.len = __shfl_sync(0xffffffffu, r.len, i);
        const long long sum = warp_count(blocks_tiles<JOINED>(p.a, p.group, o, lane, n, 32, t.longest));
        if (lane == i) t.sum = sum;
    }
    return t;
}

// Units that a key tile counts for in the 256-row kernel's work on trees, whose
// batches have blocks of up to 128 rows (one MMA tile, bound by memory) beside
// larger ones (two, bound by their chain), by turns with the requests.  us with
// 1:1, 4:5 and 7:8: 32 requests of 333-7506 keys and 17-63 tokens 130.9, 128.1,
// 127.6; of 4000 keys 127.7, 123.3, 123.6; 64 of 2-3k and 5-63 163.8, 156.7,
// 157.2; 24 of 333-16k and 9-100 147.4, 143.1, 140.3.  Either weight is better
// than none; between the two these do not decide.
// Where there are only a few tiles for every SM they count alike: ranges of
// whole tiles lie better in the blocks (one request of 64 tokens behind 4000
// keys 23.1 us, weighed 28.0).
constexpr int kTreeUnits = 8;
__device__ __forceinline__ bool light(int rows) { return rows <= kBM; }
// Tiles of a request's one block that may be light, its last, if it is.
__device__ __forceinline__ int light_tiles(const WideParams &p, const Request &r, int nb) {
    if (nb == 0 || !light(r.n * p.group.d - (nb - 1) * kRows)) return 0;
    return tiles_of<false>(p, r, nb - 1, 0);
}

// Epilogue of a row whose block has more tiles than a segment: adds O and the
// sum of the segments before, which are in the slot of a part (the block's, or
// for a whole block the one that the CTA's last block may need afterwards),
// and leaves them there for the next, or writes the block's result.
template <int D, bool BF16>
__device__ __forceinline__ void joint_epilogue(const WideParams &p, uint32_t o_col, bool valid, int slot, int more,
                                            int code, int row, size_t out_row, size_t lse_at, float m, float l_sum,
                                            float l_exact) {
    const size_t slot_at = ((size_t)blockIdx.x * 2 + (slot < 0 ? 1 : slot)) * kRows + row;
    const bool before = valid && (more & kBefore), behind = more & kBehind;
    float scale = l_sum > 0.f ? 1.0f / l_sum : 0.f, keep = 0.f;
    if (before) {
        const float m0 = p.part.slot_lse2[slot_at], l0 = p.part.slot_sum[slot_at];
        const float top = fmaxf(m, m0), ref = top == -INFINITY ? 0.f : top;
        const float a = l_exact * ex2_approx(m - ref), b = l0 * ex2_approx(m0 - ref);
        m = top;
        l_exact = a + b;
        const float inv = l_exact > 0.f ? 1.0f / l_exact : 0.f;
        scale *= a * inv;
        keep = b * inv;
    }
    const bool to_slot = behind || slot >= 0;
    float *const to_o = to_slot ? p.part.slot : p.part.plane;
    const size_t at = to_slot ? slot_at : out_row;
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t o[32];
        tmem_ld_x32(o_col + c0, o);
        tmem_ld_wait_x32(o);
#pragma unroll
        for (int q = 0; q < 32; q += 8) {
            uint32_t x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (before) ld_global_v8(x, p.part.slot + slot_at * D + c0 + q);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                o[q + k] = __float_as_uint(fmaf(__uint_as_float(x[k]), keep, __uint_as_float(o[q + k]) * scale));
        }
        if (valid && to_o) {
#pragma unroll
            for (int q = 0; q < 32; q += 8) st_global_v8(to_o + at * D + c0 + q, o + q);
        } else if (valid) {
            uint4 *const dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.a.o) + at * D + c0);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float a = __uint_as_float(o[8 * q + 2 * k]), b = __uint_as_float(o[8 * q + 2 * k + 1]);
                    w[k] = BF16 ? pack_bf16x2(a, b) : pack_f16x2(a, b);
                }
                dst[q] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        __syncwarp();  // the loads above are the whole warp's
    }
    if (!valid) return;
    if (behind) {
        p.part.slot_lse2[slot_at] = m;
        p.part.slot_sum[slot_at] = l_exact;
        return;
    }
    const float lse2 = l_exact > 0.f ? m - kWeightUnits<BF16> + log2f(l_exact) : -INFINITY;
    float *const to_lse2 = to_slot ? p.part.slot_lse2 : p.part.plane_lse2;
    if (to_lse2)
        to_lse2[at] = lse2;
    else
        p.a.lse[lse_at] = lse2 * 0.69314718055994530942f;
    if (slot != 0) p.part.code[out_row] = code ? code + part_code(0, 0, row) : 0;
}

// The part of the workspace for trees that segment g of this CTA has: words,
// and depths.
__device__ __forceinline__ size_t tree_slot(const PagedArgs &a, int g) {
    return ((size_t)blockIdx.x * 2 + (g & 1)) * a.tree_tokens;
}

// Which drafted keys the tokens of a segment see (PagedArgs), by the helpers'
// threads: each takes a token and a tile of 128 keys, walks the token's path,
// up as far as the tile begins, and sets the bits that fall into it.  The
// parents stay in L1.  Without a window the segment's first tiles are worked on
// meanwhile; under one a row needs its depth before its first.  A step up the
// path is a load that waits for the one before, and every segment walks anew:
// where tokens hang on random ones (paths of a few ln n) that does not show, on
// long paths it is what a call takes.  One request behind 333 keys, 8 heads in
// groups of 1, us with random parents, as a chain, and by the causal forward:
// 63 tokens 15, 29, 13; 256 tokens 37, 175, 17; 1024 tokens 125, 2740, 29; in
// groups of 4 19, 33, 16; 27, 79, 21; 57, 930, 33.
__device__ __forceinline__ void tree_walk(const WideParams &p, const Segment &sg, int g, int rows, int id) {
    const PagedArgs &a = p.a;
    const int t0 = sg.r0 / p.group, tokens = (sg.r0 + rows - 1) / p.group - t0 + 1;
    const int base = sg.len - sg.n, base0 = base & ~(kBN - 1);  // of the first tile
    const int tiles = (sg.key_hi - base0 + kBN - 1) / kBN;
    const int *parents = a.parents + sg.row0;
    uint4 *const words = a.tree_words + tree_slot(a, g) * a.tree_tiles;
    for (int k = id; k < tokens * tiles; k += 32 * kHelperWarps) {
        const int t = k / tiles, tile = k - t * tiles;
        const int first = base0 + tile * kBN - base;  // drafted token of the tile's first key
        const bool to_root = tile == 0 && a.window > 0;
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // keys before the drafted ones
            const int ctx = -first - 32 * q;
            w[q] = ctx <= 0 ? 0u : ctx >= 32 ? 0xFFFFFFFFu : (1u << ctx) - 1;
        }
        int depth = 0;
        for (int j = t0 + t; j >= 0 && (j >= first || to_root); ++depth) {
            const int bit = j - first;
            const uint32_t one = a.window > 0 && depth >= a.window ? 0u : 1u << (bit & 31);
#pragma unroll
            for (int q = 0; q < 4; ++q) w[q] |= bit >> 5 == q ? one : 0u;
            const int up = parents[j];
            const bool sound = up >= -1 && up < j;
            if (!sound) record_bad_args(p.status);
            j = sound ? up : -1;
        }
        words[t * a.tree_tiles + tile] = make_uint4(w[0], w[1], w[2], w[3]);
        if (to_root) a.tree_depth[tree_slot(a, g) + t] = depth - 1;
    }
}

// Of 32 keys, those from lo on and below hi.
__device__ __forceinline__ uint32_t key_bits(int lo, int hi) {
    const uint32_t from = lo <= 0 ? ~0u : lo >= 32 ? 0u : ~0u << lo;
    return hi >= 32 ? from : hi <= 0 ? 0u : from & ((1u << hi) - 1);
}

// Masks a row's 128 scores in tensor memory: all but those of keys from low to
// top that `words` (null: all) have a bit for.  A function of its own, so that
// the loop which calls it for a block's last tiles has little code for it: 64
// requests of 12 thousand keys, 32 tokens each, take 510-515 us, 527 with the
// bits tested on the scores in registers (and 502 as chains).
__device__ __noinline__ void tree_mask(uint32_t s_addr, const uint4 *words, int low, int top) {
    uint4 w = words ? *words : make_uint4(~0u, ~0u, ~0u, ~0u);
    __syncwarp();  // the loads and stores below are the whole warp's
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
        const uint32_t bits = w.x & key_bits(low - 32 * q, top - 32 * q);
        w = make_uint4(w.y, w.z, w.w, 0);
        uint32_t x[32];
        tmem_ld_x32(s_addr + 32 * q, x);
        tmem_ld_wait_x32(x);
#pragma unroll
        for (int c = 0; c < 32; ++c)
            if (!(bits >> c & 1)) x[c] = __float_as_uint(-INFINITY);
        tmem_st_x32(s_addr + 32 * q, x);
    }
    tmem_st_wait();
}

// JOINED: the shared prefix' keys are read with each request's own.  LONG: a
// block may have more tiles than a sum should.  TREE: rows hang on one another
// (PagedArgs::parents), and see of the drafted keys what their words say.
template <int D, bool BF16, bool JOINED, bool LONG, bool TREE>
__global__ void __launch_bounds__(kThreads, 1)
    paged_wide_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const WideParams p) {
    using L = WideLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::OFF_BAR);
    uint64_t *q_full = bars;
    uint64_t *k_full = q_full + 1;
    uint64_t *k_empty = k_full + L::KS;
    uint64_t *v_full = k_empty + L::KS;
    uint64_t *v_empty = v_full + L::VS;
    uint64_t *s_full = v_empty + L::VS;  // [2]
    uint64_t *p_full = s_full + 2;       // [2]
    uint64_t *o_final = p_full + 2;      // [2]
    uint64_t *seg_full = o_final + 2;    // [2]
    uint64_t *seg_empty = seg_full + 2;  // [2]
    uint64_t *q_empty = seg_empty + 2;
    uint64_t *v_clean = q_empty + 1;  // [VS]
    uint64_t *drain = v_clean + L::VS;
    uint64_t *tree_full = drain + 1;  // [2]
    Segment *segs = reinterpret_cast<Segment *>(smem + L::OFF_SEG);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::OFF_MISC + 4);
    PlanSum *sums = reinterpret_cast<PlanSum *>(smem + L::OFF_MISC + 16);
    unsigned *kept = reinterpret_cast<unsigned *>(smem + L::OFF_KEPT);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(q_full, 32 * kHelperWarps);
        mbar_init(q_empty, 1);
        for (int s = 0; s < L::VS; ++s) mbar_init(&v_clean[s], 32 * kHelperWarps);
        for (int s = 0; s < L::KS; ++s) { mbar_init(&k_full[s], 1); mbar_init(&k_empty[s], 1); }
        for (int s = 0; s < L::VS; ++s) {
            mbar_init(&v_full[s], 1);
            mbar_init(&v_empty[s], JOINED ? 1 + kHelperWarps : 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&s_full[x], 1);
            mbar_init(&p_full[x], kBM);
            mbar_init(&o_final[x], 1);
            mbar_init(&seg_full[x], 1);
            mbar_init(&seg_empty[x], 9 + kHelperWarps);  // every warp but the producer
            mbar_init(&tree_full[x], 32 * kHelperWarps);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (!p.after) wait_previous();
    launch_dependents();

    // ---------------------------------------------- the batch's units of work
    const int B = p.prefix ? 1 : p.a.B;
    {
        PlanSum sum{0, 0, 0, p.a.prefix_len, 0, 0, 0};
        auto beside = [&](const Request &r) {  // a request of the few-row kernel
            int t;
            sum.beside += pair_tiles<kFewKeys<D>>(p.a, r, t);
            if (JOINED) sum.beside += (p.a.prefix_len - prefix_low(p.a, r)) / kFewKeys<D>;
            ++sum.beside_blocks;
        };
        if (p.prefix) {
            // the few-row kernel's tiles, and the first key that any row sees
            for (int b = threadIdx.x; b < p.a.B; b += kThreads) {
                Request r;
                if (!load_request(p.a, b, r) || r.n == 0) continue;
                sum.low = min(sum.low, prefix_low(p.a, r));
                beside(r);
            }
        } else {
            for (int b = warp * 32; b < B; b += kThreads) {
                Request r{0, 0, 0};
                if (b + lane < B && !load_request(p.a, b + lane, r)) {
                    if (blockIdx.x == 0) record_bad_args(p.status);
                    r.n = 0;
                }
                if (r.n * p.group.d <= p.above) {
                    if (r.n > 0) beside(r);
                    r.n = 0;
                }
                const int nb = blocks_of(r, p.group);
                const RequestTiles tiles = request_tiles<JOINED>(p, r, nb, lane);
                sum.tiles += tiles.sum;
                if (TREE) sum.light += light_tiles(p, r, nb);
                sum.longest = max(sum.longest, tiles.longest);
                sum.blocks += nb;
                if (b + lane < kKept) kept[b + lane] = (unsigned)min(tiles.sum, (long long)kMany);
            }
        }
        sum.tiles = warp_sum(sum.tiles);
        sum.beside = warp_sum(sum.beside);
        if (TREE) sum.light = warp_sum(sum.light);
        sum.blocks = __reduce_add_sync(0xffffffffu, sum.blocks);
        sum.beside_blocks = __reduce_add_sync(0xffffffffu, sum.beside_blocks);
        sum.low = __reduce_min_sync(0xffffffffu, sum.low);
        sum.longest = __reduce_max_sync(0xffffffffu, sum.longest);
        if (lane == 0) sums[warp] = sum;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == kProducerWarp) {
        // ------------------------------------------------------ TMA producer
        if (lane == 0) {
            prefetch_tmap(&tm_q);
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_v);
        }
        Request whole{0, 0, p.a.prefix_len};  // the prefix pass: one request of all rows
        WideWork work{0, 0};
        long long few_tiles = 0, few_pairs = 0;
        int most = gridDim.x, prefix_lo = p.a.prefix_len, longest = 0;
        long long light_all = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            work.tiles += (long long)sums[w].tiles * p.a.Hkv;
            work.blocks += (long long)sums[w].blocks * p.a.Hkv;
            few_tiles += (long long)sums[w].beside * p.a.Hkv;
            few_pairs += (long long)sums[w].beside_blocks * p.a.Hkv;
            prefix_lo = min(prefix_lo, sums[w].low);
            longest = max(longest, sums[w].longest);
            if (TREE) light_all += (long long)sums[w].light * p.a.Hkv;
        }
        if (p.prefix) {
            whole.n = end_row(p.a);
            work = prefix_work(p.a, whole.n, p.group.d, prefix_lo);
        }
        if (p.shared && few_pairs > 0) most = min(most, wide_sms(work.units(), few_tiles, few_pairs));
        // Whole blocks only, each by the CTA in whose range it begins: a cut
        // one costs the merge of its parts, and a segment more in most CTAs
        // once there are more tiles than CTAs; a whole one leaves others idle
        // for what it takes longer than they do.  Measured, us, cut and whole:
        //   a CTA for each block: 32 blocks of 1 or 2 tiles 18.2 and 16.3, 64
        //     of 1-4 26.8 and 21.3, of 7 24.2 and 22.4; with as many CTAs as
        //     tiles 16 of 1-4 17.4 and 19.2, else 32 of 7 or 8 24.5 and 27.5
        //   several blocks a CTA: 256 of 1-4 36.9 and 34.5, 512 of 4 70 and
        //     63, 256 of 8 57.8 and 49.5, 640 of 1-10 91.9 and 90.8, 512 of
        //     12 118.7 and 121.4, 256 of 1-16 55.2 and 68.9
        const long long loaded = work.tiles + work.blocks * kBlockCost;
        const bool spare = work.blocks <= most;
        const int uncut = !p.prefix && longest > 1 &&
                          (!spare              ? longest <= 10
                           : work.tiles > most ? (2ll * longest - 7) * most <= 2 * loaded
                                               : longest <= 2);
        // from one lane: the compiler then sees one value for the warp (0.5 %)
        const bool by_blocks = __shfl_sync(0xffffffffu, uncut, 0);
        // units of a tile, and how many fewer a light block's has
        const int unit = TREE ? __shfl_sync(0xffffffffu, work.tiles > 4 * kSms ? kTreeUnits : 1, 0) : 1;
        const int less = unit > 1 ? 1 : 0;
        const int cost = (by_blocks ? kBlockCost : work.block_cost()) * unit;
        const long long T = (by_blocks ? loaded : work.units()) * unit - light_all * less;
        // a range of so many units has a tile's first one in it, wherever it lies in a block
        const int G = (int)min((long long)most, max(1ll, T / unit));
        const Ranges ranges(T, G);
        const int page_keys = min(1 << p.a.shift, kBN);
        const int box_bytes = page_keys * 128;
        const int half = lane % L::NBOX, sub = lane / L::NBOX;
        const bool boxed = lane < L::NBOX * (kBN / page_keys);
        const int c = blockIdx.x;
        const long long u0 = c < G ? ranges.start(c) : T, u1 = c < G ? ranges.start(c + 1) : T;
        int nk = 0, nv = 0, ns = 0;  // K and V tiles and segments handed on
        bool ok = true;
        // hands a segment to the other warps
        auto tell = [&](const Segment &sg) {
            const int slot = ns & 1;
            const bool got = ns < 2 || mbar_wait(&seg_empty[slot], ((ns >> 1) + 1) & 1, abort_flag, p.status, 39);
            ok = __all_sync(0xffffffffu, got);
            if (ok && lane == 0) {
                segs[slot] = sg;
                mbar_arrive(&seg_full[slot]);
            }
            ++ns;
        };
        // A tree's keys are read by one CTA, once, where its rows fit a block
        // and its pages are its own: evicted first, they leave L2 to the parts
        // that the merge reads (32 requests of 17-63 tokens 127.8 us and 122.8,
        // 64 of 8-16k keys 528 and 519; all of one size as long as their chains
        // again).  Pages that requests share are read once by each holder, at
        // about the same time, and lose nothing: 8, 15 and 32 branches of 32
        // tokens behind one prompt of 16k keys 102, 176 and 348 us without,
        // 100, 172 and 344; of 64k keys 341, 640 and 1302, and 336, 631, 1289.
        const uint64_t once = l2_evict_first();
        bool read_once = false;
        auto load_box = [&](void *dst, const CUtensorMap *tm, uint64_t *bar, int row, int plane) {
            if (TREE && read_once)
                tma_load_3d_hint(dst, tm, bar, half * 64, row, plane, once);
            else
                tma_load_3d(dst, tm, bar, half * 64, row, plane);
        };
        auto load = [&](int b, Request &r) -> bool {
            if (!p.prefix) return load_request(p.a, b, r) && r.n * p.group.d > p.above;
            r = whole;
            return r.n > 0;
        };
        // the request that holds unit u0, and its first unit
        int b = 0;
        long long base = 0;
        if (u0 < u1 && !p.prefix) {
            for (; b < B; b += 32) {
                Request r{0, 0, 0};
                if (b + lane < B && !load(b + lane, r)) r.n = 0;
                const int nb = blocks_of(r, p.group);
                const unsigned held = b >= kKept ? kMany : b + lane < B ? kept[b + lane] : 0;
                long long tiles = held;
                if (__any_sync(0xffffffffu, held == kMany)) tiles = request_tiles<JOINED>(p, r, nb, lane).sum;
                if (TREE) tiles = tiles * unit - light_tiles(p, r, nb) * less;
                const long long units = (tiles + (long long)nb * cost) * p.a.Hkv;
                long long incl = units;
#pragma unroll
                for (int s = 1; s < 32; s <<= 1) {
                    const long long x = __shfl_up_sync(0xffffffffu, incl, s);
                    if (lane >= s) incl += x;
                }
                const unsigned past = __ballot_sync(0xffffffffu, base + incl > u0);
                if (past) {
                    const int k = __ffs(past) - 1;
                    base += __shfl_sync(0xffffffffu, incl - units, k);
                    b += k;
                    break;
                }
                base += __shfl_sync(0xffffffffu, incl, 31);
            }
        }
        long long u = u0;
        bool fresh = true;  // the place within the request is still to be found
        int hk = 0, blk = 0;
        long long blk0 = base;  // first unit of (hk, blk)
        for (; ok && u < u1 && b < B; ++b, fresh = false, hk = 0, blk = 0) {
            Request r;
            if (!load(b, r)) continue;
            const int nb = blocks_of(r, p.group);
            read_once = TREE && nb == 1;
            if (fresh) {
                long long tiles = (long long)nb * range_tiles(prefix_lo, r.len);
                if (!p.prefix && b < kKept && kept[b] != kMany) {
                    tiles = kept[b];
                } else if (!p.prefix) {
                    Request mine{0, 0, 0};
                    if (lane == 0) mine = r;
                    tiles = __shfl_sync(0xffffffffu, request_tiles<JOINED>(p, mine, lane == 0 ? nb : 0, lane).sum, 0);
                }
                if (TREE) tiles = tiles * unit - light_tiles(p, r, nb) * less;
                const long long per_head = tiles + (long long)nb * cost;
                hk = (int)((u - base) / per_head);
                blk0 = base + (long long)hk * per_head;
                // the block of that head: 32 at a time
                for (blk = 0; blk < nb; blk += 32) {
                    using Count = std::conditional_t<TREE, long long, int>;  // 32 blocks' tiles, but not units, fit 32 bits
                    Count units = 0;
                    if (blk + lane < nb) {
                        units = tiles_of<JOINED>(p, r, blk + lane, prefix_lo);
                        if (TREE) units *= unit - (light(r.n * p.group.d - (blk + lane) * kRows) ? less : 0);
                        units += cost;
                    }
                    Count incl = units;
#pragma unroll
                    for (int s = 1; s < 32; s <<= 1) {
                        const Count x = __shfl_up_sync(0xffffffffu, incl, s);
                        if (lane >= s) incl += x;
                    }
                    const unsigned past = __ballot_sync(0xffffffffu, blk0 + incl > u);
                    if (past) {
                        const int k = __ffs(past) - 1;
                        blk0 += __shfl_sync(0xffffffffu, incl - units, k);
                        blk += k;
                        break;
                    }
                    blk0 += __shfl_sync(0xffffffffu, incl, 31);
                }
            }
            const int *own_table = p.prefix ? p.a.prefix_pages : p.a.block_table + (size_t)b * p.a.max_pages;
            for (; ok && hk < p.a.Hkv && u < u1; ++hk, blk = 0) {
                for (; ok && blk < nb && u < u1; ++blk) {
                    Segment sg;
                    sg.row0 = r.row0;
                    sg.n = r.n;
                    sg.len = r.len;
                    sg.r0 = blk * kRows;
                    sg.hk = hk;
                    block_keys(p, r, blk, prefix_lo, sg.key_lo, sg.key_hi);
                    sg.front = block_front<JOINED>(p, r, blk, sg.front_lo);
                    const int nt = sg.front + range_tiles(sg.key_lo, sg.key_hi);
                    const long long tile0 = blk0 + cost;  // unit of its first tile
                    const bool begun = blk0 < u0;  // in the range of the CTA before
                    // a tile of several units belongs to the CTA that has the first one
                    const int w = TREE && light(r.n * p.group.d - sg.r0) ? unit - less : unit;
                    const int first = by_blocks ? 0 : (int)((max(0ll, u - tile0) + w - 1) / w);
                    const int end =
                        !by_blocks ? (int)((min((long long)nt * w, u1 - tile0) + w - 1) / w) : begun ? 0 : nt;
                    blk0 = tile0 + (long long)nt * w;
                    u = u1 < blk0 ? u1 : blk0;
                    if (end <= first) continue;  // the range ends before the block's first tile
                    const bool is_whole = first == 0 && end == nt;
                    sg.j0 = first;
                    sg.nj = end - first;
                    sg.slot = is_whole ? -1 : first == 0 ? 1 : 0;
                    // a block that goes on in the next CTA belongs to the one it began in
                    sg.code = sg.slot == 1 ? part_code(ranges.owner(blk0 - w) - c + 1, c, 0) : 0;
                    sg.more = sg.pad[0] = sg.pad[1] = 0;
                    auto load_tiles = [&] {
                        tell(sg);
                        for (int i = 0; ok && i < sg.nj; ++i) {
                            // pages that hold no key of the block's range are not looked up
                            const KeyTile<JOINED> tile(sg, i, p.a.prefix_len);
                            const int *table = tile.in_front ? p.a.prefix_pages : own_table;
                            const int key0 = tile.kv0 + sub * page_keys;
                            const bool live = boxed && key0 < tile.hi && key0 + page_keys > tile.lo;
                            int page = 0;
                            if (live) {
                                page = table[key0 >> p.a.shift];
                                if (page < 0 || page >= p.a.num_pages) {
                                    record_bad_args(p.status);
                                    page = p.a.num_pages;  // out of the tensor: the copy fills zeros
                                }
                            }
                            const int bytes = __popc(__ballot_sync(0xffffffffu, live)) * box_bytes;
                            const int in_page = key0 & ((1 << p.a.shift) - 1);
                            const int ks = nk % L::KS, vs = nv % L::VS;
                            bool got =
                                nk < L::KS || mbar_wait(&k_empty[ks], ((nk / L::KS) + 1) & 1, abort_flag, p.status, 31);
                            if (!(ok = __all_sync(0xffffffffu, got))) break;
                            if (lane == 0) mbar_arrive_expect_tx(&k_full[ks], bytes);
                            __syncwarp();
                            if (live)
                                load_box(smem + L::OFF_K + ks * L::TILE + half * L::BOX + sub * box_bytes, &tm_k,
                                         &k_full[ks], in_page, page * p.a.Hkv + hk);
                            ++nk;
                            got = nv < L::VS ||
                                  mbar_wait(&v_empty[vs], ((nv / L::VS) + 1) & 1, abort_flag, p.status, 32);
                            if (!(ok = __all_sync(0xffffffffu, got))) break;
                            if (lane == 0) mbar_arrive_expect_tx(&v_full[vs], bytes);
                            __syncwarp();
                            if (live)
                                load_box(smem + L::OFF_V + vs * L::TILE + half * L::BOX + sub * box_bytes, &tm_v,
                                         &v_full[vs], in_page, page * p.a.Hkv + hk);
                            ++nv;
                        }
                    };
                    if (!LONG) {
                        load_tiles();
                        continue;
                    }
                    for (; ok && sg.j0 < end; sg.j0 += kMaxTiles<BF16>) {
                        sg.nj = min(end - sg.j0, kMaxTiles<BF16>);
                        sg.more = (sg.j0 > first ? kBefore : 0) | (sg.j0 + sg.nj < end ? kBehind : 0);
                        load_tiles();
                    }
                }
            }
        }
        if (ok) {
            Segment sg{};
            sg.nj = -1;
            tell(sg);
        }
        if (!ok && lane == 0) {
            // given up: let copies in flight land before the CTA exits
            for (int i = max(0, nk - L::KS); i < nk; ++i)
                mbar_wait_drain(&k_full[i % L::KS], (i / L::KS) & 1, 10000000ull);
            for (int i = max(0, nv - L::VS); i < nv; ++i)
                mbar_wait_drain(&v_full[i % L::VS], (i / L::VS) & 1, 10000000ull);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // -------------------------------------------------------- MMA issuer
        if (lane == 0) {
            constexpr uint32_t fmt = BF16 ? 1u : 0u;
            constexpr uint32_t idesc_s = make_idesc(kBM, kBN, fmt, false, false);
            constexpr uint32_t idesc_pv = make_idesc(kBM, D, fmt, false, true);
            const uint64_t q_desc0 = make_sdesc_sw128(smem_u32(smem + L::OFF_Q), 16, 1024);
            const uint64_t k_desc0 = make_sdesc_sw128(smem_u32(smem + L::OFF_K), 16, 1024);
            const uint64_t v_desc0 = make_sdesc_sw128(smem_u32(smem + L::OFF_V), L::BOX, 1024);
            // u counts K/V tiles over all segments, first: a segment's first tile
            auto issue_s = [&](int x, int u) {
                const uint64_t q_desc = sdesc_advance(q_desc0, x * L::TILE);
                const uint64_t k_desc = sdesc_advance(k_desc0, (u % L::KS) * L::TILE);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = (kk >> 2) * L::BOX + (kk & 3) * 32;
                    mma_f16_ss(tmem + kColS + x * 128, sdesc_advance(q_desc, off), sdesc_advance(k_desc, off), idesc_s,
                               kk > 0 ? 1u : 0u);
                }
                mma_commit(&s_full[x]);
            };
            auto issue_pv = [&](int x, int u, bool first) {
                const uint64_t v_desc = sdesc_advance(v_desc0, (u % L::VS) * L::TILE);
                const uint32_t p_col = tmem + kColS + x * 128;
#pragma unroll
                for (int kk = 0; kk < kBN / 16; ++kk)
                    mma_f16_ts(tmem + kColO + x * 128, p_col + kk * 8, sdesc_advance(v_desc, kk * 2048), idesc_pv,
                               (!first || kk > 0) ? 1u : 0u);
            };
            auto wait = [&](uint64_t *bar, int parity, int site) -> bool {
                const bool got = mbar_wait(bar, parity, abort_flag, p.status, site);
                tc_fence_after();
                return got;
            };
            bool ok = true;
            int u = 0, step_b = 0;  // tiles of all segments; of those that have a tile B
            uint32_t cleans = 0;    // a bit per V stage: parity of its clears
            for (int g = 0; ok; ++g) {
                if (!(ok = wait(&seg_full[g & 1], (g >> 1) & 1, 40))) break;
                const Segment sg = segs[g & 1];
                const int nj = sg.nj;
                const bool two = sg.n * p.group.d - sg.r0 > kBM;
                mbar_arrive(&seg_empty[g & 1]);
                if (nj < 0) break;
                if (!(ok = wait(q_full, g & 1, 33) && wait(&k_full[u % L::KS], (u / L::KS) & 1, 34))) break;
                issue_s(0, u);
                if (two) issue_s(1, u);
                mma_commit(&k_empty[u % L::KS]);
                if (nj == 1) mma_commit(q_empty);
                // V of the segment's first tile
                if (!(ok = wait(&v_full[u % L::VS], (u / L::VS) & 1, 35))) break;
                for (int i = 0; i < nj; ++i, ++u) {
                    const int vs = u % L::VS, kn = (u + 1) % L::KS, vn = (u + 1) % L::VS;
                    const bool last = i + 1 == nj;
                    if (KeyTile<JOINED>(sg, i, p.a.prefix_len).hides()) {
                        if (!(ok = wait(&v_clean[vs], cleans >> vs & 1, 42))) break;
                        cleans ^= 1u << vs;
                    }
                    if (!(ok = wait(&p_full[0], u & 1, 36))) break;
                    issue_pv(0, u, i == 0);
                    if (last) {
                        mma_commit(&o_final[0]);
                    } else {
                        if (!(ok = wait(&k_full[kn], ((u + 1) / L::KS) & 1, 34))) break;
                        issue_s(0, u + 1);
                        if (!two) {
                            mma_commit(&k_empty[kn]);
                            if (i + 2 == nj) mma_commit(q_empty);
                        }
                    }
                    if (two) {
                        if (!(ok = wait(&p_full[1], step_b & 1, 36))) break;
                        ++step_b;
                        issue_pv(1, u, i == 0);
                        if (last) mma_commit(&o_final[1]);
                    }
                    mma_commit(&v_empty[vs]);
                    if (last) continue;
                    if (!(ok = wait(&v_full[vn], ((u + 1) / L::VS) & 1, 35))) break;
                    if (two) {
                        issue_s(1, u + 1);
                        mma_commit(&k_empty[kn]);
                        if (i + 2 == nj) mma_commit(q_empty);
                    }
                }
            }
            // every MMA issued above has completed once `drain` flips
            mma_commit(drain);
            mbar_wait_drain(drain, 0, 100000000ull);
        }
        __syncwarp();
    } else if (warp >= kMmaWarp + 1) {
        // ------------------------------------------------------------ helpers
        const int id = threadIdx.x - 32 * (kMmaWarp + 1);
        constexpr int CH = D / 8, STEP = 32 * kHelperWarps / CH;  // 16-byte pieces of a row; rows a pass
        bool ok = true;
        int u = 0, boxed_q = -1;  // tiles of the segments before; last segment whose Q came by TMA
        for (int g = 0; ok; ++g) {
            bool got = mbar_wait(&seg_full[g & 1], (g >> 1) & 1, abort_flag, p.status, 43);
            if (!__all_sync(0xffffffffu, got)) break;
            const Segment sg = segs[g & 1];
            __syncwarp();
            if (lane == 0) mbar_arrive(&seg_empty[g & 1]);
            if (sg.nj < 0) break;
            // Q into the operand layout, a row's pieces by neighbouring lanes,
            // once the last S of the segment before has read its own; rows
            // past the block's are zeros
            got = g == 0 || mbar_wait(q_empty, (g - 1) & 1, abort_flag, p.status, 44);
            if (!__all_sync(0xffffffffu, got)) break;
            const int rows = min(sg.n * p.group.d - sg.r0, kRows);
            if (p.q_box) {
                // whole tokens fill a tile: one box per tile and 64 columns.
                // Rows past the block's are the next request's, or zeros: they
                // touch no other row and are never written.
                boxed_q = g;
                if (id == 0) {
                    const int tiles = rows > kBM ? 2 : 1, tok = sg.row0 + sg.r0 / p.group;
                    mbar_arrive_expect_tx(q_full, tiles * L::TILE);
                    for (int x = 0; x < tiles; ++x)
                        for (int bx = 0; bx < L::NBOX; ++bx)
                            tma_load_4d(smem + L::OFF_Q + x * L::TILE + bx * L::BOX, &tm_q, q_full, bx * 64, 0, sg.hk,
                                        tok + x * p.q_box);
                } else {
                    mbar_arrive(q_full);
                }
            } else {
                const int ch = id % CH;
                const int t0 = sg.r0 / p.group, h0 = sg.r0 - t0 * p.group.d;
                const uint4 *src =
                    static_cast<const uint4 *>(p.a.q) + ((size_t)(sg.row0 + t0) * p.a.Hq + sg.hk * p.group.d) * CH + ch;
#pragma unroll 8
                for (int r = id / CH; r < kRows; r += STEP) {
                    uint8_t *dst = smem + L::OFF_Q + (r >> 7) * L::TILE + (ch >> 3) * L::BOX + (r & 127) * 128 +
                                   (((ch & 7) ^ (r & 7)) << 4);
                    const int t = (h0 + r) / p.group, h = h0 + r - t * p.group.d;
                    if (r < rows)
                        cp_async_16(smem_u32(dst), src + ((size_t)t * p.a.Hq + h) * CH);
                    else
                        *reinterpret_cast<uint4 *>(dst) = make_uint4(0, 0, 0, 0);
                }
                cp_async_wait_all();
                fence_proxy_async_smem();
                mbar_arrive(q_full);
            }
            if (TREE) {
                // the segment two before has been seen by all: the last S of
                // the one before, just waited for, comes behind its last P
                tree_walk(p, sg, g, rows, id);
                mbar_arrive(&tree_full[g & 1]);
                __syncwarp();
            }
            // V rows that no row of the block sees may hold anything (the rest
            // of a page, a buffer that was not filled), and 0 * NaN is NaN:
            // clear them in the tiles that have some, the first and the last
            // of each sequence.  The wait for a tile must not take an earlier
            // filling of its buffer for it: where a prefix ends amid the
            // tiles, a buffer is refilled only after the helpers have seen
            // what it held; else the last tile is waited for when the last S
            // of the segment is through, as the one that the buffer held
            // before has arrived then.
            for (int i = 0; ok && i < sg.nj; i += JOINED ? 1 : max(1, sg.nj - 1)) {
                const KeyTile<JOINED> tile(sg, i, p.a.prefix_len);
                const int vs = (u + i) % L::VS;
                if (!JOINED) {
                    if (!tile.hides()) continue;
                    got = i == 0 || mbar_wait(q_empty, g & 1, abort_flag, p.status, 46);
                    if (!(ok = __all_sync(0xffffffffu, got))) break;
                }
                got = mbar_wait(&v_full[vs], ((u + i) / L::VS) & 1, abort_flag, p.status, 45);
                if (!(ok = __all_sync(0xffffffffu, got))) break;
                if (tile.hides()) {
                    uint4 *v = reinterpret_cast<uint4 *>(smem + L::OFF_V + vs * L::TILE);
                    for (int k = id; k < kBN * 8 * L::NBOX; k += 32 * kHelperWarps) {
                        const int key = tile.kv0 + ((k >> 3) & (kBN - 1));
                        if (key < tile.lo || key >= tile.hi) v[k] = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(&v_clean[vs]);
                    __syncwarp();
                }
                if (JOINED && lane == 0) mbar_arrive(&v_empty[vs]);
            }
            u += sg.nj;
        }
        // a Q that is still in flight, if the others gave up, lands before the CTA exits
        if (id == 0 && boxed_q >= 0) mbar_wait_drain(q_full, boxed_q & 1, 10000000ull);
        __syncwarp();
    } else {
        // ------------------------------------------------ softmax + epilogue
        const int x = warp >> 2;
        const int quarter = warp & 3;
        const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t col_s = kColS + x * 128, col_o = kColO + x * 128;
        const int row = threadIdx.x;
        const float sl2 = p.scale_log2;
        auto next_segment = [&](int g, Segment &sg) -> bool {
            const bool got = mbar_wait(&seg_full[g & 1], (g >> 1) & 1, abort_flag, p.status, 41);
            if (!__all_sync(0xffffffffu, got)) return false;
            sg = segs[g & 1];
            __syncwarp();
            if (lane == 0) mbar_arrive(&seg_empty[g & 1]);
            return true;
        };
        Segment sg;
        int step = 0, finals = 0;  // tiles of this warpgroup's Q tile, and segments that had it
        bool ok = next_segment(0, sg);
        for (int g = 0; ok && sg.nj >= 0; ++g) {
            // this thread's row: where it is and which keys it sees
            const int rows = min(sg.n * p.group.d - sg.r0, kRows);
            const bool two = rows > kBM, active = x == 0 || two, valid = row < rows;
            int tok = 0, head = 0, hi = 0x7FFFFFFF, lo = -0x7FFFFFFF;
            int tree_at = 0;  // TREE: of the row's token in the workspace
            auto tree_low = [&]() {  // first key before the drafted ones (below hi) that the row sees
                return p.a.window > 0 && valid ? min(window_low(hi + p.a.tree_depth[tree_at] + 1, p.a.window), hi)
                                               : -0x7FFFFFFF;
            };
            auto wait_tree = [&]() -> bool {
                const bool got = mbar_wait(&tree_full[g & 1], (g >> 1) & 1, abort_flag, p.status, 47);
                return __all_sync(0xffffffffu, got);
            };
            if (TREE && active && p.a.window > 0 && !(ok = wait_tree())) break;
            if (valid) {
                const int t = (sg.r0 + row) / p.group;
                head = sg.hk * p.group.d + (sg.r0 + row) - t * p.group.d;
                tok = sg.row0 + t;
                if (p.prefix) {
                    const int b = request_of(p.a, tok);
                    Request r;
                    if (load_request(p.a, b, r)) {
                        hi = p.a.prefix_len + r.len - r.n + (tok - r.row0) + 1;
                        lo = p.a.window > 0 ? window_low(hi, p.a.window) : 0;
                    }
                } else {
                    // no window: below every place (a prefix' first key is at -prefix_len)
                    hi = sg.len - sg.n + t + 1;
                    lo = p.a.window > 0 ? window_low(hi, p.a.window) : -0x7FFFFFFF;
                    if constexpr (TREE) {
                        tree_at = (int)tree_slot(p.a, g) + t - sg.r0 / p.group;
                        hi = sg.len - sg.n;
                    }
                }
            }
            const int nj = sg.nj;
            float m_ref = -INFINITY;
            float l_sum = 0.0f;    // sum of the rounded P fed to the MMA: normalises O
            float l_exact = 0.0f;  // sum of the unrounded P: gives L
            const int hi_w = __reduce_min_sync(0xffffffffu, hi);
            const int lo_w = __reduce_max_sync(0xffffffffu, TREE ? tree_low() : lo);
            for (int u = 0; ok && active && u < nj; ++u, ++step) {
                const bool got_s = mbar_wait(&s_full[x], step & 1, abort_flag, p.status, 37);
                if (!__all_sync(0xffffffffu, got_s)) { ok = false; break; }
                tc_fence_after();
                const uint32_t s_addr = lane_base + col_s;
                const KeyTile<JOINED> tile(sg, u, p.a.prefix_len);
                const int shift = tile.in_front ? p.a.prefix_len : 0;  // the tile's keys as places
                const int kv0 = tile.kv0 - shift, key_lo = tile.lo - shift, key_hi = tile.hi - shift;
                const bool hides = kv0 + kBN > min(hi_w, key_hi) || kv0 < max(lo_w, key_lo);  // uniform in the warp
                if (TREE && hides) {
                    if (!(ok = wait_tree())) break;
                    const uint4 *words = p.a.tree_words + tree_at * p.a.tree_tiles + (kv0 >> 7) - (hi >> 7);  // kBN keys
                    const bool drafted = valid && kv0 + kBN > hi && kv0 < key_hi;
                    tree_mask(s_addr, drafted ? words : nullptr, max(tree_low(), key_lo) - kv0, key_hi - kv0);
                }
                uint32_t s[128];
                tmem_ld_x32(s_addr + 0, s + 0);
                tmem_ld_x32(s_addr + 32, s + 32);
                tmem_ld_x32(s_addr + 64, s + 64);
                tmem_ld_x32(s_addr + 96, s + 96);
                tmem_ld_wait_x32(s + 0);
                tmem_ld_wait_x32(s + 32);
                tmem_ld_wait_x32(s + 64);
                tmem_ld_wait_x32(s + 96);
                if (!TREE && hides) {
                    const int top = min(hi, key_hi), low = max(lo, key_lo);
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (kv0 + c >= top || kv0 + c < low) s[c] = __float_as_uint(-INFINITY);
                }
                float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
                for (int c = 0; c < 128; c += 8) {
                    mx0 = fmax3(mx0, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
                    mx1 = fmax3(mx1, __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
                    mx2 = fmax3(mx2, __uint_as_float(s[c + 4]), __uint_as_float(s[c + 5]));
                    mx3 = fmax3(mx3, __uint_as_float(s[c + 6]), __uint_as_float(s[c + 7]));
                }
                const float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * sl2;
                float alpha = 1.0f;
                bool rescale = false;
                if (mx > m_ref + kRescaleThreshold) {
                    alpha = ex2_approx(m_ref - mx);  // 0 on the first visible tile
                    l_sum *= alpha;
                    l_exact *= alpha;
                    m_ref = mx;
                    rescale = true;
                }
                __syncwarp();
                const float m_use = m_ref == -INFINITY ? 0.0f : m_ref;  // nothing seen yet: P = 0
                const float2 neg_m = make_float2(kWeightUnits<BF16> - m_use, kWeightUnits<BF16> - m_use);
                const float2 sl2x2 = make_float2(sl2, sl2);
                float2 lr01 = make_float2(0.f, 0.f), lr23 = lr01, le01 = lr01, le23 = lr01;
                constexpr int CH = 32;
#pragma unroll
                for (int hh = 0; hh < 128 / CH; ++hh) {
                    uint32_t pk[CH / 2];
#pragma unroll
                    for (int c = CH * hh; c < CH * hh + CH; c += 4) {
                        const float2 x01 =
                            ffma2(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sl2x2, neg_m);
                        const float2 x23 =
                            ffma2(make_float2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), sl2x2, neg_m);
                        const float p0 = ex2_approx(x01.x), p1 = ex2_approx(x01.y);
                        const float p2 = ex2_approx(x23.x), p3 = ex2_approx(x23.y);
                        const int k = (c - CH * hh) / 2;
                        if constexpr (BF16) {
                            pk[k] = pack_bf16x2(p0, p1);
                            pk[k + 1] = pack_bf16x2(p2, p3);
                            lr01 = add_bf16x2_f32x2(pk[k], lr01);
                            lr23 = add_bf16x2_f32x2(pk[k + 1], lr23);
                        } else {
                            pk[k] = pack_f16x2_sat(p0, p1);
                            pk[k + 1] = pack_f16x2_sat(p2, p3);
                            lr01 = fadd2(lr01, unpack2<BF16>(pk[k]));
                            lr23 = fadd2(lr23, unpack2<BF16>(pk[k + 1]));
                        }
                        le01 = fadd2(le01, make_float2(p0, p1));
                        le23 = fadd2(le23, make_float2(p2, p3));
                    }
                    tmem_st_x16(lane_base + col_s + 16 * hh, pk);
                }
                l_sum += (lr01.x + lr01.y) + (lr23.x + lr23.y);
                l_exact += (le01.x + le01.y) + (le23.x + le23.y);
                if (u >= 1 && __any_sync(0xffffffffu, rescale)) {
                    uint32_t o[D];
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += 32) tmem_ld_x32(lane_base + col_o + c0, o + c0);
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += 32) tmem_ld_wait_x32(o + c0);
#pragma unroll
                    for (int c = 0; c < D; c += 2) {
                        const float2 r = fmul2(make_float2(__uint_as_float(o[c]), __uint_as_float(o[c + 1])),
                                               make_float2(alpha, alpha));
                        o[c] = __float_as_uint(r.x);
                        o[c + 1] = __float_as_uint(r.y);
                    }
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += 32) tmem_st_x32(lane_base + col_o + c0, o + c0);
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&p_full[x]);
            }
            if (active) {
                const bool got = ok && mbar_wait(&o_final[x], finals & 1, abort_flag, p.status, 38);
                ++finals;
                ok = __all_sync(0xffffffffu, got);
                tc_fence_after();
            }
            if (!ok) break;
            if (LONG && active && sg.more) {
                const size_t out_row = (size_t)tok * p.a.Hq + head;
                joint_epilogue<D, BF16>(p, lane_base + col_o, valid, sg.slot, sg.more, sg.code, row, out_row,
                                        (size_t)head * p.a.total + tok, m_ref, l_sum, l_exact);
                tc_fence_before();
            } else if (active) {
                const float inv_l = l_sum > 0.f ? 1.0f / l_sum : 0.f;
                const size_t out_row = (size_t)tok * p.a.Hq + head;
                // whole blocks are final, or go to the plane to be merged with
                // the other pass'; parts go to their slot
                float *to_o = p.part.plane, *to_lse2 = p.part.plane_lse2;
                size_t at = out_row;
                if (sg.slot >= 0) {
                    to_o = p.part.slot;
                    to_lse2 = p.part.slot_lse2;
                    at = ((size_t)blockIdx.x * 2 + sg.slot) * kRows + row;
                }
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t o[32];
                    tmem_ld_x32(lane_base + col_o + c0, o);
                    tmem_ld_wait_x32(o);
#pragma unroll
                    for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * inv_l);
                    if (valid && to_o) {
                        float *dst = to_o + at * D + c0;
#pragma unroll
                        for (int q = 0; q < 4; ++q) st_global_v8(dst + 8 * q, o + 8 * q);  // whole sectors
                    } else if (valid) {
                        uint16_t *dst = static_cast<uint16_t *>(p.a.o) + at * D + c0;
                        uint32_t w[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float a = __uint_as_float(o[2 * k]), b = __uint_as_float(o[2 * k + 1]);
                            w[k] = BF16 ? pack_bf16x2(a, b) : pack_f16x2(a, b);
                        }
                        if (p.o32) {
                            st_global_v8(dst, w);
                            st_global_v8(dst + 16, w + 8);
                        } else {
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                reinterpret_cast<uint4 *>(dst)[q] =
                                    make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
                        }
                    }
                    __syncwarp();  // the loads above are the whole warp's
                }
                if (valid) {
                    const float lse2 = l_exact > 0.f ? m_ref - kWeightUnits<BF16> + log2f(l_exact) : -INFINITY;
                    if (to_lse2)
                        to_lse2[at] = lse2;
                    else
                        p.a.lse[(size_t)head * p.a.total + tok] = lse2 * 0.69314718055994530942f;
                    if (sg.slot != 0) p.part.code[out_row] = sg.code ? sg.code + part_code(0, 0, row) : 0;
                }
                // the reads of O above come before the MMAs that a later arrive permits
                tc_fence_before();
            }
            ok = next_segment(g + 1, sg);
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    // the merge, which waits for this kernel, then also has the other pass'
    wait_previous();
}

template <int D, bool BF16>
cudaError_t launch_wide_t(const PagedArgs &a, const PagedPlan &w, bool prefix, bool after, cudaStream_t st) {
    using L = WideLayout<D>;
    CUtensorMap tq, tk, tv;
    if (!make_tmap_pages(&tk, a.k_cache, BF16, D, a.page_size, a.num_pages, a.Hkv, kBN) ||
        !make_tmap_pages(&tv, a.v_cache, BF16, D, a.page_size, a.num_pages, a.Hkv, kBN))
        return cudaErrorInvalidValue;
    WideParams p;
    p.a = a;
    const int g = a.Hq / a.Hkv;
    p.group = fast_div(g);
    p.q_box = kBM % g == 0 ? kBM / g : 0;
    if (!make_tmap_rows(&tq, a.q, BF16, D, g, a.Hkv, a.total, p.q_box ? p.q_box : 1)) return cudaErrorInvalidValue;
    p.prefix = prefix ? 1 : 0;
    p.shared = prefix ? w.few : w.mixed;
    p.above = w.mixed ? kMaxRows : 0;
    p.after = after ? 1 : 0;
    p.o32 = (reinterpret_cast<uintptr_t>(a.o) & 31u) == 0;
    p.part = prefix ? w.prefix : w.own;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.status = device_status_ptr();
    // under a window a block of a tree's rows may see as many more keys as there are drafted ones
    const long long tiles = prefix ? w.prefix_tiles : w.own_tiles + (a.parents ? a.max_new / kWideKeys + 1 : 0);
    const bool many = tiles > kMaxTiles<BF16>;
    auto kernel = many ? paged_wide_kernel<D, BF16, false, true, false> : paged_wide_kernel<D, BF16, false, false, false>;
    if (w.joined)
        kernel = many ? paged_wide_kernel<D, BF16, true, true, false> : paged_wide_kernel<D, BF16, true, false, false>;
    if (a.parents)
        kernel = many ? paged_wide_kernel<D, BF16, false, true, true> : paged_wide_kernel<D, BF16, false, false, true>;
    return launch_after(kernel, p.part.ctas, kThreads, L::ALLOC, st, tq, tk, tv, p);
}

}  // namespace

cudaError_t launch_paged_wide(const PagedArgs &a, const PagedPlan &w, bool prefix, bool after, cudaStream_t st) {
    if (a.d == 128)
        return a.bf16 ? launch_wide_t<128, true>(a, w, prefix, after, st)
                      : launch_wide_t<128, false>(a, w, prefix, after, st);
    return a.bf16 ? launch_wide_t<64, true>(a, w, prefix, after, st)
                  : launch_wide_t<64, false>(a, w, prefix, after, st);
}

}  // namespace fa
