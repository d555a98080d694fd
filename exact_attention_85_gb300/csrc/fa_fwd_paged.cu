// fa_fwd_paged.cu -- forward attention from a paged key/value cache for
// requests with few query rows (decoding, drafted tokens).
//
// Row i of request b (n_b new rows, len_b keys of its own, of which the last
// n_b belong to the rows) stands at place p = len_b - n_b + i and sees its
// own keys max(0, p - W + 1) .. p.  The n_b * g rows that read one key/value
// head (g = Hq / Hkv query heads share it), 16 at most, are worked on
// together: [V2] section 6.1 with the running maximum and sum of the softmax,
// the maximum moved only when a score passes it by more than 8 (log2 units),
// as in the dense forward.
//
// Few rows make the products narrow, so they are formed transposed, with the
// keys (S^T = K Q^T) and the head's columns (O~^T += V^T P^T) as the long side
// of the warp-level MMA and 8 query rows as its short one: half the
// instructions of the other way for up to 8 rows.  Measured, reading from L2
// (one CTA alone) and from memory (42 to 72 SMs): 49 and 54 GB/s an SM with
// the rows on the long side, 59 and 73 this way.  All SMs together are bound
// by reading the cache: 461 us for 64 requests of 8-16k keys (453 on another
// card), 7.0 TB/s where a copy, which writes as well, reaches 6.8.  Everything
// else here serves to keep copies in flight.
//
// Work is cut into units of one tile of keys (32 KB of K and V).  All units
// of all (request, key/value head) pairs are numbered in order and every CTA
// takes an equal, contiguous range, so a batch of any mixture of lengths
// keeps every SM reading to the end; a CTA's range covers the end of one
// pair, some whole pairs and the beginning of another.  Whole pairs are
// written out directly; the parts of a pair that several CTAs share go to
// the workspace as (O~ / l, log2 sum) and a second kernel merges them (with a
// shared prefix that has a pass of its own, everything does, and is merged
// with that pass' results; a short prefix is simply the first tiles of every
// pair here).
//   warps 0-3  each a quarter of every tile's keys, all rows; their four
//              results are merged through the last tile's buffer
//   warps 4, 5 producers of K and of V: each plans the CTA's range, reads the
//              block-table entries and starts one TMA copy per page (the 16
//              of a tile of 16-key pages at d = 64 took one warp 1.06 us, two
//              0.87); the first also copies Q, and describes each tile to the
//              others
#include "../../include/fa.h"
#include "host_util.h"
#include "mma_sync.cuh"
#include "paged.h"
#include "paged_dev.cuh"
#include "ptx.cuh"

namespace fa {

namespace {

constexpr int kConsumers = 4;  // warps
constexpr int kFewWarps = kConsumers + 2;  // and two producers
constexpr int kFewThreads = 32 * kFewWarps;
// Two CTAs per SM.  us with 190, 212, 250 and 304 CTAs: 64 requests of 8-16k
// keys 462, 456, 458, 461; 32 of 333-7506 87.8, 83.5, 80.8, 83.0; beside the
// 256-row kernel 256 requests on a 16k prefix 202 with any, 64 on 8k 44.3,
// 45.5, 48.5, 48.4 on a card where the whole call takes 48, and no difference
// on one where it takes 44.
constexpr int kMaxCtas = 2 * kSms;
constexpr int kStages = 3;
constexpr int kMinUnits = 2;   // units a CTA takes at least
// A pair costs its tiles and about as much as one more (Q, the merge of the
// warps, the stores), counted when ranges are cut.
constexpr int kPairCost = 1;
constexpr float kMoveBy = 8.0f;  // log2 units by which a score passes the maximum before that moves

enum : int { kFirst = 1, kLast = 2, kMask = 4, kPart = 8, kSlot1 = 16, kFront = 32 };

// What the producer tells the consumers about a tile.
struct TileInfo {
    int row0, n, len, kv0;
    int hk, flags;
    int code;  // of the pair's rows, but for the row number (PartView)
    int pad;
};

template <int D>
struct FewLayout {
    static constexpr int TK = kFewKeys<D>;          // keys per tile
    static constexpr int KW = TK / kConsumers;      // keys per warp and tile
    static constexpr int TILE = TK * D * 2;         // K or V
    static constexpr int QBYTES = kMaxRows * D * 2;
    static constexpr int OFF_Q = kStages * 2 * TILE;
    static constexpr int OFF_INFO = OFF_Q + kStages * QBYTES;
    static constexpr int OFF_TREE = OFF_INFO + kStages * (int)sizeof(TileInfo);  // [kStages][16]
    static constexpr int OFF_BAR = OFF_TREE + kStages * kMaxRows * 4;
    static constexpr int OFF_ML = OFF_BAR + 2 * kStages * 8;           // [3][4 warps][16]
    static constexpr int OFF_MISC = OFF_ML + 3 * kConsumers * 16 * 4;  // abort flag, the warps' sums
    static constexpr int BYTES = OFF_MISC + 16 + kFewWarps * (int)sizeof(PlanSum);
    static constexpr int ALLOC = BYTES + 1024;
    static_assert(2 * (ALLOC + 1024) <= 228 * 1024, "two CTAs per SM");
    static_assert(kConsumers * kMaxRows * D * 4 <= 2 * TILE, "the merge fits one stage");
};

struct FewParams {
    PagedArgs a;
    FastDiv group;  // query heads per key/value head
    float scale_log2;
    unsigned int *status;
    PartView part;
    int whole;  // a unit is a whole pair, not a tile
    int after;  // runs beside the call's kernel before, which has waited for what came before
    int mixed;  // requests of more rows are the 256-row kernel's
    int joined; // the shared prefix' keys are read with each request's own
};

// A request of this kernel: one with rows, and no more than it takes.
__device__ __forceinline__ bool few_request(const FewParams &p, int b, Request &r) {
    return load_request(p.a, b, r) && r.n > 0 && r.n * p.group.d <= kMaxRows;
}

// First tile and number of tiles of the shared prefix that a request's rows
// see, where they are read with its own.
template <int TK>
__device__ __forceinline__ int front_tiles(const FewParams &p, const Request &r, int &t0) {
    const int lo = p.joined ? prefix_low(p.a, r) : 0;
    t0 = lo / TK;
    return p.joined && lo < p.a.prefix_len ? (p.a.prefix_len + TK - 1) / TK - t0 : 0;
}

// All tiles of a pair of request r.
template <int TK>
__device__ __forceinline__ int all_tiles(const FewParams &p, const Request &r) {
    int t0;
    const int front = front_tiles<TK>(p, r, t0);
    return front + pair_tiles<TK>(p.a, r, t0);
}

// The paths of a tree of up to 16 drafted tokens, one a lane: the tokens from
// which lane i's hangs down, itself among them, a bit each, but for those that
// a window hides, and its depth above them.  Twice as many with every step.
__device__ __forceinline__ uint32_t tree_paths(const FewParams &p, const Request &r, int lane) {
    int up = lane < r.n ? p.a.parents[r.row0 + lane] : -1;
    if (up < -1 || up >= lane) {
        record_bad_args(p.status);
        up = -1;
    }
    uint32_t path = 1u << lane;
#pragma unroll
    for (int s = 1; s < kMaxRows; s *= 2) {
        const int from = up < 0 ? lane : up;
        const uint32_t more = __shfl_sync(0xffffffffu, path, from);
        const int next = __shfl_sync(0xffffffffu, up, from);
        if (up >= 0) path |= more;
        up = up < 0 ? -1 : next;
    }
    path &= 0xFFFFu;  // of lanes that have no token
    const int depth = __popc(path) - 1;
    // the lowest are the farthest
    for (int out = depth + 1 - p.a.window; p.a.window > 0 && out > 0; --out) path &= path - 1;
    return path | (uint32_t)depth << 16;
}

// NT: 8-row groups of a pair (rows up to 8 * NT).  TREE: rows hang on one
// another (PagedArgs::parents).
template <int D, bool BF16, int NT, bool TREE>
__global__ void __launch_bounds__(kFewThreads, 2)
    paged_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const FewParams p) {
    using L = FewLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::OFF_BAR), *empty = full + kStages;
    TileInfo *info = reinterpret_cast<TileInfo *>(smem + L::OFF_INFO);
    uint32_t *tree = reinterpret_cast<uint32_t *>(smem + L::OFF_TREE);
    float *sm_m = reinterpret_cast<float *>(smem + L::OFF_ML);  // [4][16], then l, then exact l
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::OFF_MISC);
    PlanSum *sums = reinterpret_cast<PlanSum *>(smem + L::OFF_MISC + 16);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int B = p.a.B, Hkv = p.a.Hkv;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 34);  // the bytes of K, of V, and 32 lanes' shares of Q
            mbar_init(&empty[s], kConsumers);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (!p.after) wait_previous();
    launch_dependents();
    {   // tiles of the whole batch
        PlanSum sum{0, 0, 0, p.a.prefix_len, 0, 0, 0};
        for (int b = threadIdx.x; b < B; b += kFewThreads) {
            Request r;
            if (!load_request(p.a, b, r)) {
                if (blockIdx.x == 0) record_bad_args(p.status);
                continue;
            }
            if (r.n == 0) continue;
            if (r.n * p.group.d <= kMaxRows) {
                sum.tiles += all_tiles<L::TK>(p, r);
                ++sum.blocks;
            } else {
                int blocks;
                sum.beside += block_tiles(p.a, r, p.group.d, blocks);
                if (p.joined) sum.beside += (long long)blocks * ((p.a.prefix_len - prefix_low(p.a, r)) / kWideKeys);
                sum.beside_blocks += blocks;
            }
            sum.low = min(sum.low, prefix_low(p.a, r));
        }
        sum.tiles = warp_sum(sum.tiles);
        sum.blocks = __reduce_add_sync(0xffffffffu, sum.blocks);
        sum.low = __reduce_min_sync(0xffffffffu, sum.low);
        if (p.mixed) {
            sum.beside = warp_sum(sum.beside);
            sum.beside_blocks = __reduce_add_sync(0xffffffffu, sum.beside_blocks);
        }
        if (lane == 0) sums[warp] = sum;
    }
    __syncthreads();

    if (warp >= kConsumers) {
        // ----------------------------------------------------------- producers
        const bool first_one = warp == kConsumers;
        const CUtensorMap *tm = first_one ? &tm_k : &tm_v;
        if (lane == 0) prefetch_tmap(tm);
        long long tiles = 0, pairs = 0;
        WideWork beside{0, 0};
        int low = p.a.prefix_len, most = gridDim.x;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
            tiles += (long long)sums[w].tiles * Hkv;
            pairs += (long long)sums[w].blocks * Hkv;
            beside.tiles += (long long)sums[w].beside * Hkv;
            beside.blocks += (long long)sums[w].beside_blocks * Hkv;
            low = min(low, sums[w].low);
        }
        // the kernel beside this one has some of the SMs to itself
        if (!p.mixed && !p.joined && p.a.prefix_len > 0) beside = prefix_work(p.a, end_row(p.a), p.group.d, low);
        if (beside.blocks > 0)
            most = min(most, 2 * (kSms - wide_sms(beside.units(), tiles, pairs)));
        const long long T = p.whole ? pairs : tiles + pairs * kPairCost;
        const int G = (int)min((long long)most, max(1ll, p.whole ? T : T / kMinUnits));
        const Ranges ranges(T, G);
        const int c = blockIdx.x;
        const long long u0 = c < G ? ranges.start(c) : T, u1 = c < G ? ranges.start(c + 1) : T;
        // the request that holds unit u0
        int b = 0;
        long long base = 0;  // first unit of request b
        if (u0 < u1) {
            for (; b < B; b += 32) {
                Request r;
                long long units = 0;
                if (b + lane < B && few_request(p, b + lane, r))
                    units = (p.whole ? 1ll : (long long)all_tiles<L::TK>(p, r) + kPairCost) * Hkv;
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
        // this lane's box: a page of the tile, its 64-column halves one behind
        // the other (128-byte swizzled rows)
        const int page_keys = min(1 << p.a.shift, L::TK);
        const int box_bytes = page_keys * D * 2;
        // A request's own keys are read by one CTA only, unless requests share
        // pages.  A joined prefix' are read with every request's own; the
        // policy is the same for them.
        const uint64_t once = l2_evict_first();
        const int sub = lane;
        const bool boxed = sub < L::TK / page_keys;
        uint8_t *const tiles_at = smem + (first_one ? 0 : L::TILE);
        int st = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        long long u = u0;
        while (ok && u < u1 && b < B) {
            Request r;
            if (!few_request(p, b, r)) {
                ++b;
                continue;
            }
            int front0, own0;  // first tiles
            const int front = front_tiles<L::TK>(p, r, front0), nt = front + pair_tiles<L::TK>(p.a, r, own0);
            const int cost = p.whole ? 0 : kPairCost, per_pair = p.whole ? 1 : nt + cost;  // units
            const uint32_t paths = TREE && first_one ? tree_paths(p, r, lane) : 0;
            int hk = (int)((u - base) / per_pair);
            for (; ok && hk < Hkv && u < u1; ++hk) {
                const long long pair0 = base + (long long)hk * per_pair, tile0 = pair0 + cost;
                const int j0 = (int)max(0ll, u - tile0), j1 = p.whole ? nt : (int)min((long long)nt, u1 - tile0);
                u = u1 < pair0 + per_pair ? u1 : pair0 + per_pair;
                if (j1 <= j0) continue;  // the range ends before the pair's first tile
                const bool whole = j0 == 0 && j1 == nt;
                // a pair that goes on in the next CTA belongs to the one it began in
                const int code =
                    !whole && j0 == 0 ? part_code(ranges.owner(pair0 + per_pair - 1) - c + 1, c, 0) : 0;
                for (int j = j0; j < j1; ++j) {
                    // the prefix' tiles come first; places count from its start
                    const bool in_front = j < front;
                    const int kv0 = (in_front ? front0 + j : own0 + j - front) * L::TK;
                    const int shift = in_front ? p.a.prefix_len : 0, end = in_front ? p.a.prefix_len : r.len;
                    const int lo_min = p.a.window > 0 ? max(0, r.len - r.n + 1 - p.a.window + shift) : 0;
                    const int lo_max = p.a.window > 0 ? max(0, r.len - p.a.window + shift) : 0;
                    const int hi_min = min(end, r.len - r.n + (TREE ? 0 : 1) + shift);
                    const int *table = in_front ? p.a.prefix_pages : p.a.block_table + (size_t)b * p.a.max_pages;
                    // pages that hold no visible key are neither looked up nor read
                    const int key0 = kv0 + sub * page_keys;
                    const bool live = boxed && key0 < end && key0 + page_keys > lo_min;
                    int page = 0;
                    if (live) {
                        page = table[key0 >> p.a.shift];
                        if (page < 0 || page >= p.a.num_pages) {
                            record_bad_args(p.status);
                            page = p.a.num_pages;  // out of the tensor: the copy fills zeros
                        }
                    }
                    const int boxes = __popc(__ballot_sync(0xffffffffu, live));
                    const bool got = issued < kStages || mbar_wait(&empty[st], phase ^ 1, abort_flag, p.status, 21);
                    if (!__all_sync(0xffffffffu, got)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0 && first_one) {
                        TileInfo t;
                        t.row0 = r.row0;
                        t.n = r.n;
                        t.len = r.len;
                        t.kv0 = kv0;
                        t.hk = hk;
                        t.code = code;
                        t.flags = (j == j0 ? kFirst : 0) | (j + 1 == j1 ? kLast : 0) |
                                  (kv0 < lo_max || kv0 + L::TK > hi_min ? kMask : 0) | (whole ? 0 : kPart) |
                                  (j0 == 0 ? kSlot1 : 0) | (in_front ? kFront : 0);
                        info[st] = t;
                    }
                    if (TREE && first_one && j == j0) {
                        if (lane < kMaxRows) tree[st * kMaxRows + lane] = paths;
                        __syncwarp();
                    }
                    if (lane == 0) mbar_arrive_expect_tx(&full[st], boxes * box_bytes);
                    __syncwarp();
                    if (live)
                        tma_load_4d_hint(tiles_at + st * 2 * L::TILE + sub * box_bytes, tm, &full[st], 0,
                                         key0 & ((1 << p.a.shift) - 1), 0, page * Hkv + hk, once);
                    if (first_one && j == j0) {
                        // Q rows of the pair: row r is head r % g of token r / g
                        constexpr int CH = D / 8;  // 16-byte pieces of a row
                        const int rows = r.n * p.group.d;
                        for (int i = lane; i < rows * CH; i += 32) {
                            const int row = i / CH, ch = i % CH;
                            const int t = row / p.group;
                            const uint4 *src =
                                static_cast<const uint4 *>(p.a.q) +
                                ((size_t)(r.row0 + t) * p.a.Hq + hk * p.group.d + (row - t * p.group.d)) * CH + ch;
                            cp_async_16(smem_u32(smem + L::OFF_Q + st * L::QBYTES) + row * (D * 2) +
                                            ((ch ^ (row & 7)) << 4),
                                        src);
                        }
                    }
                    if (first_one) cp_async_arrive(&full[st]);
                    ++issued;
                    if (++st == kStages) {
                        st = 0;
                        phase ^= 1;
                    }
                }
            }
            if (hk == Hkv) {
                base += (long long)per_pair * Hkv;
                ++b;
            }
        }
        if (!ok && lane == 0) {
            // let copies in flight land before the CTA exits
            for (int i = max(0, issued - kStages); i < issued; ++i)
                mbar_wait_drain(&full[i % kStages], (i / kStages) & 1, 10000000ull);
        }
        if (lane == 0) {
            // a tile that ends the stream
            const bool got = !ok || issued < kStages || mbar_wait(&empty[st], phase ^ 1, abort_flag, p.status, 22);
            if (ok && got) {
                if (first_one) info[st].flags = -1;
                mbar_arrive_expect_tx(&full[st], 0);
            }
        }
        __syncwarp();
        if (ok && first_one) cp_async_arrive(&full[st]);
    } else {
        // ----------------------------------------------------------- consumers
        const int quad = lane & 3, rw = lane >> 2;  // this lane's keys rw, rw + 8; rows 2 quad, + 1
        constexpr int MT = L::KW / 16;              // 16-key groups of this warp
        // byte offsets of the lane's ldmatrix rows: pages lie one behind the
        // other in a tile, the halves of a page's rows likewise
        const int page_shift = min(p.a.shift, D == 128 ? 6 : 7);
        const int half_bytes = 128 << page_shift;
        auto row_at = [&](int key) {
            return (key >> page_shift) * (D / 64 * half_bytes) + (key & ((1 << page_shift) - 1)) * 128;
        };
        int k_at[MT], v_at[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            k_at[i] = row_at(warp * L::KW + i * 16 + ((lane >> 3) & 1) * 8 + (lane & 7));
            v_at[i] = row_at(warp * L::KW + i * 16 + (lane >> 4) * 8 + (lane & 7));
        }
        const uint32_t k_swz = ((lane >> 4) ^ (lane & 7)) << 4, v_swz = (((lane >> 3) & 1) ^ (lane & 7)) << 4;
        uint32_t qf[NT][D / 16][2];
        float acc[NT][D / 16][4];  // columns rw, rw + 8 of each 16; rows 2 quad, + 1
        float m[NT][2], l[NT][2], le[NT][2];
        int hi[NT][2], lo[NT][2];
        uint32_t path[NT][2];  // TREE: drafted keys that the row sees; it sees all before hi as far as lo
        int st = 0;
        uint32_t phase = 0;
        for (;;) {
            bool ok = mbar_wait(&full[st], phase, abort_flag, p.status, 23);
            ok = __all_sync(0xffffffffu, ok);
            TileInfo t;
            t.flags = 0;
            if (ok) {
                t = info[st];
                if (t.flags == -1) break;
            } else {
                // every warp reaches the barrier below once per pair, so that
                // none is left waiting there
                named_bar_and(1, kConsumers * 32, false);
                break;
            }
            const uint32_t ks = smem_u32(smem + st * 2 * L::TILE), vs = ks + L::TILE;
            if (t.flags & kFirst) {
                // rows past the pair's own hold whatever the buffer held: they
                // touch no other row and are never written
                const uint32_t qs = smem_u32(smem + L::OFF_Q + st * L::QBYTES);
#pragma unroll
                for (int g = 0; g < NT; ++g) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; kk += 2) {
                        uint32_t f[4];
                        const int row = g * 8 + (lane & 7);
                        ldmatrix_x4(f, qs + row * (D * 2) + (((2 * kk + (lane >> 3)) ^ (row & 7)) << 4));
                        qf[g][kk][0] = f[0];
                        qf[g][kk][1] = f[1];
                        qf[g][kk + 1][0] = f[2];
                        qf[g][kk + 1][1] = f[3];
                    }
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) acc[g][i][0] = acc[g][i][1] = acc[g][i][2] = acc[g][i][3] = 0.f;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        m[g][x] = -INFINITY;
                        l[g][x] = le[g][x] = 0.f;
                        const int token = (g * 8 + quad * 2 + x) / p.group;
                        int depth = token;
                        if constexpr (TREE) {
                            const uint32_t seen = tree[st * kMaxRows + min(token, kMaxRows - 1)];
                            path[g][x] = seen & 0xFFFFu;
                            depth = seen >> 16;
                        }
                        hi[g][x] = t.len - t.n + depth + 1;
                        // no window: below every place (a prefix' first key is at -prefix_len)
                        lo[g][x] = p.a.window > 0 ? hi[g][x] - p.a.window : -0x7FFFFFFF;
                        if (TREE) hi[g][x] = t.len - t.n;
                    }
                }
            }
            // S^T: this warp's KW keys
            const int w0 = warp * L::KW;
            float s[MT][NT][4];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
#pragma unroll
                for (int g = 0; g < NT; ++g) s[i][g][0] = s[i][g][1] = s[i][g][2] = s[i][g][3] = 0.f;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t kf[4];
                    ldmatrix_x4(kf, ks + k_at[i] + (kk >> 2) * half_bytes + (((kk & 3) << 5) ^ k_swz));
#pragma unroll
                    for (int g = 0; g < NT; ++g) mma_16x8x16<BF16>(s[i][g], kf, qf[g][kk][0], qf[g][kk][1]);
                }
            }
            // the tile's keys end here, and places of its keys begin there
            const int end = t.flags & kFront ? p.a.prefix_len : t.len, shift = t.flags & kFront ? p.a.prefix_len : 0;
            if (t.flags & kMask) {
#pragma unroll
                for (int i = 0; i < MT; ++i) {
#pragma unroll
                    for (int g = 0; g < NT; ++g) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = t.kv0 + w0 + i * 16 + rw + (e >> 1) * 8;
                            const int place = key - shift;
                            bool hidden = key >= end || place < lo[g][e & 1];
                            if constexpr (TREE) {
                                // a drafted key is seen on the row's path, whatever its place
                                if (key < end && place >= hi[g][e & 1])
                                    hidden = !(path[g][e & 1] >> ((place - hi[g][e & 1]) & 15) & 1);
                            } else {
                                hidden |= place >= hi[g][e & 1];
                            }
                            if (hidden) s[i][g][e] = -INFINITY;
                        }
                    }
                }
            }
            // the maximum of a row moves when a score passes it by 8
            float mx[NT][2];
            bool passed = false;
#pragma unroll
            for (int g = 0; g < NT; ++g) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float v = fmaxf(s[0][g][x], s[0][g][x + 2]);
                    if (MT == 2) v = fmax3(v, s[MT - 1][g][x], s[MT - 1][g][x + 2]);
                    mx[g][x] = v * p.scale_log2;
                    passed |= mx[g][x] > m[g][x] + kMoveBy;
                }
            }
            if (__any_sync(0xffffffffu, passed)) {
#pragma unroll
                for (int g = 0; g < NT; ++g) {
                    float alpha[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float v = mx[g][x];
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                        alpha[x] = 1.f;
                        if (v > m[g][x] + kMoveBy) {
                            alpha[x] = ex2_approx(m[g][x] - v);  // 0 for the first visible score
                            m[g][x] = v;
                        }
                        l[g][x] *= alpha[x];
                        le[g][x] *= alpha[x];
                    }
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        acc[g][i][0] *= alpha[0];
                        acc[g][i][1] *= alpha[1];
                        acc[g][i][2] *= alpha[0];
                        acc[g][i][3] *= alpha[1];
                    }
                }
            }
            // P, rounded to the 16-bit type and turned into P^T; l sums the
            // rounded P that the MMA reads (O~ / l is then an exactly
            // normalised mix of V rows), le the unrounded ones (LSE)
            uint32_t pf[MT][NT][2];
#pragma unroll
            for (int g = 0; g < NT; ++g) {
                // a row that has seen nothing yet keeps -inf: 0 stands in for it
                const float n0 = m[g][0] == -INFINITY ? 0.f : kWeightUnits<BF16> - m[g][0];
                const float n1 = m[g][1] == -INFINITY ? 0.f : kWeightUnits<BF16> - m[g][1];
#pragma unroll
                for (int i = 0; i < MT; ++i) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float a = ex2_approx(fmaf(s[i][g][2 * y], p.scale_log2, n0));
                        const float c = ex2_approx(fmaf(s[i][g][2 * y + 1], p.scale_log2, n1));
                        const uint32_t pk = BF16 ? pack_bf16x2(a, c) : pack_f16x2_sat(a, c);
                        const float2 w = unpack2<BF16>(pk);
                        l[g][0] += w.x;
                        l[g][1] += w.y;
                        le[g][0] += a;
                        le[g][1] += c;
                        pf[i][g][y] = transpose_8x8(pk);
                    }
                }
            }
            // O~^T += V^T P^T
            const int k_end = end - t.kv0 - w0;  // keys of this warp that exist
            const int k_low = p.a.window > 0 ? t.len - t.n + 1 - p.a.window + shift - t.kv0 - w0 : 0;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    uint32_t vf[4];
                    ldmatrix_x4_trans(vf, vs + v_at[i] + (j >> 2) * half_bytes + (((j & 3) << 5) ^ v_swz));
                    if (t.flags & kMask) {
                        // what no row sees may hold anything, and 0 * NaN is NaN
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int k0 = i * 16 + (e >> 1) * 8 + quad * 2;
                            if (k0 >= k_end || k0 < k_low) vf[e] &= 0xFFFF0000u;
                            if (k0 + 1 >= k_end || k0 + 1 < k_low) vf[e] &= 0x0000FFFFu;
                        }
                    }
                    // a product of its own, added in fp32: as an addend of the
                    // next product the sum would lose up to 2^-26 of itself to
                    // every term, which the tensor cores cut down to its bits
                    // (64 requests of a million keys, values of mean 1: 1.0e-3,
                    // where storing fp16 makes 2.2e-4)
#pragma unroll
                    for (int g = 0; g < NT; ++g) {
                        float t[4] = {0.f, 0.f, 0.f, 0.f};
                        mma_16x8x16<BF16>(t, vf, pf[i][g][0], pf[i][g][1]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[g][j][e] += t[e];
                    }
                }
            }
            if (t.flags & kLast) {
                // merge the four warps' results through this tile's buffer
                constexpr int ROWS = 8 * NT;
#pragma unroll
                for (int g = 0; g < NT; ++g) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
#pragma unroll
                        for (int d = 4; d < 32; d *= 2) {
                            l[g][x] += __shfl_xor_sync(0xffffffffu, l[g][x], d);
                            le[g][x] += __shfl_xor_sync(0xffffffffu, le[g][x], d);
                        }
                    }
                }
                if (!named_bar_and(1, kConsumers * 32, true)) break;  // all warps have read the tile
                float *buf = reinterpret_cast<float *>(smem + st * 2 * L::TILE) + warp * (ROWS * D);
#pragma unroll
                for (int g = 0; g < NT; ++g) {
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int row = g * 8 + quad * 2 + (e & 1), col = i * 16 + rw + (e >> 1) * 8;
                            buf[row * D + (col ^ (quad << 3))] = acc[g][i][e];  // exchanged by row: no bank conflicts
                        }
                    }
                    if (rw == 0) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int at = warp * 16 + g * 8 + quad * 2 + x;
                            sm_m[at] = m[g][x];
                            sm_m[kConsumers * 16 + at] = l[g][x];
                            sm_m[2 * kConsumers * 16 + at] = le[g][x];
                        }
                    }
                }
                named_bar_sync(2, kConsumers * 32);
                // several threads a row, four neighbouring columns at a time
                constexpr int TPR = kConsumers * 32 / ROWS;
                const int row = threadIdx.x / TPR, part = threadIdx.x % TPR;
                if (row < t.n * p.group.d) {
                    float top = -INFINITY, sum = 0.f, exact = 0.f, f[kConsumers];
#pragma unroll
                    for (int w = 0; w < kConsumers; ++w) top = fmaxf(top, sm_m[w * 16 + row]);
                    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
                    for (int w = 0; w < kConsumers; ++w) {
                        f[w] = ex2_approx(sm_m[w * 16 + row] - ref);
                        sum += f[w] * sm_m[kConsumers * 16 + w * 16 + row];
                        exact += f[w] * sm_m[2 * kConsumers * 16 + w * 16 + row];
                    }
                    const float inv = sum > 0.f ? 1.f / sum : 0.f;
                    const float lse2 = exact > 0.f ? top - kWeightUnits<BF16> + log2f(exact) : -INFINITY;
                    const float *from = reinterpret_cast<const float *>(smem + st * 2 * L::TILE) + row * D;
                    const int tok = row / p.group;
                    const int h = t.hk * p.group.d + row - tok * p.group.d;
                    const size_t out_row = (size_t)(t.row0 + tok) * p.a.Hq + h;
                    // a whole pair's result is final, or goes to the plane to be
                    // merged with the shared prefix'; a part goes to its slot
                    float *to_o = p.part.plane, *to_lse2 = p.part.plane_lse2;
                    size_t at = out_row;
                    if (t.flags & kPart) {
                        to_o = p.part.slot;
                        to_lse2 = p.part.slot_lse2;
                        at = ((size_t)blockIdx.x * 2 + (t.flags & kSlot1 ? 1 : 0)) * kMaxRows + row;
                    }
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += TPR * 4) {
                        const int c = c0 + part * 4;
                        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int w = 0; w < kConsumers; ++w) {
                            const float4 x = *reinterpret_cast<const float4 *>(from + w * (ROWS * D) +
                                                                               (c ^ (((row >> 1) & 3) << 3)));
                            o.x = fmaf(f[w], x.x, o.x);
                            o.y = fmaf(f[w], x.y, o.y);
                            o.z = fmaf(f[w], x.z, o.z);
                            o.w = fmaf(f[w], x.w, o.w);
                        }
                        o.x *= inv;
                        o.y *= inv;
                        o.z *= inv;
                        o.w *= inv;
                        if (to_o) {
                            *reinterpret_cast<float4 *>(to_o + at * D + c) = o;
                        } else {
                            const uint2 w = BF16 ? make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w))
                                                 : make_uint2(pack_f16x2(o.x, o.y), pack_f16x2(o.z, o.w));
                            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.a.o) + out_row * D + c) = w;
                        }
                    }
                    if (part == 0) {
                        if (to_lse2)
                            to_lse2[at] = lse2;
                        else
                            p.a.lse[(size_t)h * p.a.total + t.row0 + tok] = lse2 * 0.69314718055994530942f;
                        if (!p.whole && (!(t.flags & kPart) || (t.flags & kSlot1)))
                            p.part.code[out_row] =
                                t.code ? t.code + part_code(0, 0, row) + (p.mixed ? kFewCode : 0) : 0;
                    }
                }
                fence_proxy_async_smem();  // the buffer's next writer is a TMA copy
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
            if (++st == kStages) {
                st = 0;
                phase ^= 1;
            }
        }
    }
    // the merge, which waits for this kernel, then also has the prefix' results
    wait_previous();
}

// Merges the parts of every row that has several.  A lane has C columns of a
// row.  C = 8 (32 bytes of a part, 16 of O): a warp works on 2 rows (d = 128)
// or 4, and W warps share the parts of their rows, each taking every W-th: one
// where there are many rows, with few parts each, eight where there are few
// rows that can have many.  C = 16 from 16 thousand rows on, twice the rows a
// warp: what it waits for is two rounds of loads, codes and then parts (up to
// four or two in flight, and the next rows' codes), and what it issues is
// mostly addresses and weights, the same for 16 columns as for 8.  (A call of
// 65 thousand rows, most of two parts: 147 us with 8 columns, 144 with 16; one
// of 8192 rows with some eight: 200.5 and 203.  A row a warp, 4 columns a
// lane, took the merge of the first from 12 us to 25.)
struct MergeParams {
    PagedArgs a;
    PartView own, prefix, beside;
    FastDiv heads;  // Hq
    int warps;      // W
};

constexpr int kMergeWarps = 8;

// Parts of a row by its code.  An unsound request's codes are not written, so
// a code is held to the slots that there are.
__device__ __forceinline__ int parts_of(const PartView &v, int code) {
    const int pieces = code & kMaxPieces, cta = code >> 9 & kMaxPieces, slot_row = code >> 18 & 255;
    if (code == 0) return v.plane ? 1 : 0;
    return pieces < 2 || cta + pieces > v.ctas || slot_row >= v.slot_rows ? 0 : pieces;
}

// PREFIX: the rows have a shared prefix' parts as well.  C: columns a lane.
template <int D, bool BF16, bool PREFIX, int C>
__global__ void __launch_bounds__(32 * kMergeWarps, 3) paged_merge_kernel(const MergeParams p) {
    constexpr int LPR = D / C, RPW = 32 / LPR;  // lanes of a row, rows of a warp
    constexpr int U = 32 / C;
    constexpr bool SHARED = C == 8;  // several warps may share a row's parts
    __shared__ float sm_o[SHARED ? kMergeWarps : 1][32][9], sm_top[kMergeWarps][32], sm_sum[kMergeWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = (lane % LPR) * C;
    const int W = SHARED ? p.warps : 1, sub = warp % W;
    const int rows = p.a.total * p.a.Hq;  // 31 bits, as the entry points see to
    wait_previous();
    launch_dependents();
    // rows behind the batch's have no part
    const long long id_lo = (long long)first_row(p.a) * p.a.Hq, id_hi = (long long)end_row(p.a) * p.a.Hq;
    const long long step = (long long)gridDim.x * (kMergeWarps / W) * RPW;
    long long id = ((long long)blockIdx.x * (kMergeWarps / W) + warp / W) * RPW + lane / LPR;
    int next_own = 0, next_pre = 0;
    auto load_codes = [&](long long i) {
        if (i >= rows) return;
        next_own = p.own.code[i];
        if (PREFIX) next_pre = p.prefix.code[i];
    };
    load_codes(id);
    // the same number of rounds for every warp of a block: there is a barrier
    for (long long first = (long long)blockIdx.x * (kMergeWarps / W) * RPW; first < rows; first += step, id += step) {
        const int c_own = next_own, c_pre = next_pre;
        load_codes(id + step);
        int n_own = 0, n_all = 0;
        if (id >= id_lo && id < id_hi) {
            n_own = parts_of(c_own & kFewCode ? p.beside : p.own, c_own);
            n_all = n_own + (PREFIX ? parts_of(p.prefix, c_pre) : 0);
        }
        float acc[C], top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int e = 0; e < C; ++e) acc[e] = 0.f;
        // where the parts of a pass begin: piece k is at one plane row, or two slots further each
        auto locate = [&](const PartView &v, int code, const float *&lse2, const float *&o, size_t &stride) {
            const size_t at =
                code ? ((size_t)(code >> 9 & kMaxPieces) * 2 + 1) * v.slot_rows + (code >> 18 & 255) : (size_t)id;
            lse2 = (code ? v.slot_lse2 : v.plane_lse2) + at;
            o = (code ? v.slot : v.plane) + at * D + col;
            stride = v.slot_rows;
        };
        const float *lse_own, *o_own, *lse_pre = nullptr, *o_pre = nullptr;
        size_t stride_own, stride_pre = 0;
        locate(c_own & kFewCode ? p.beside : p.own, c_own, lse_own, o_own, stride_own);
        if (PREFIX) locate(p.prefix, c_pre, lse_pre, o_pre, stride_pre);
        for (int k0 = sub; k0 < n_all; k0 += W * U) {
            float lse2[U];
            uint32_t x[U][C];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int k = k0 + i * W;
                lse2[i] = -INFINITY;
                if (k >= n_all) continue;
                const bool own = !PREFIX || k < n_own;
                const int piece = own ? k : k - n_own;
                // piece 0 in slot 1 of its CTA, the others in slot 0 of the next ones
                const size_t off = piece ? (size_t)(2 * piece - 1) * (own ? stride_own : stride_pre) : 0;
                lse2[i] = (own ? lse_own : lse_pre)[off];
                const float *o = (own ? o_own : o_pre) + off * D;
#pragma unroll
                for (int q = 0; q < C; q += 8) ld_global_v8(x[i] + q, o + q);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (lse2[i] == -INFINITY) continue;
                const float to = fmaxf(top, lse2[i]);
                const float a = ex2_approx(top - to), w = ex2_approx(lse2[i] - to);
                sum = fmaf(sum, a, w);
#pragma unroll
                for (int e = 0; e < C; ++e) acc[e] = fmaf(acc[e], a, w * __uint_as_float(x[i][e]));
                top = to;
            }
        }
        if (SHARED && W > 1) {
#pragma unroll
            for (int e = 0; e < C; ++e) sm_o[warp][lane][e] = acc[e];
            sm_top[warp][lane] = top;
            sm_sum[warp][lane] = sum;
            __syncthreads();
            for (int k = 1; sub == 0 && k < W; ++k) {
                const float t2 = sm_top[warp + k][lane];
                if (t2 == -INFINITY) continue;
                const float to = fmaxf(top, t2);
                const float a = ex2_approx(top - to), w = ex2_approx(t2 - to);
                sum = sum * a + w * sm_sum[warp + k][lane];
#pragma unroll
                for (int e = 0; e < C; ++e) acc[e] = acc[e] * a + w * sm_o[warp + k][lane][e];
                top = to;
            }
            __syncthreads();
        }
        if (n_all == 0 || sub) continue;  // final already, a row of no request, or another warp's to write
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        uint32_t w[C / 2];
#pragma unroll
        for (int e = 0; e < C / 2; ++e)
            w[e] = BF16 ? pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv)
                        : pack_f16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
        uint4 *const to = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.a.o) + (size_t)id * D + col);
#pragma unroll
        for (int q = 0; q < C / 8; ++q) to[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
        if (col == 0) {
            const int tok = (int)id / p.heads, h = (int)id - tok * p.a.Hq;
            p.a.lse[(size_t)h * p.a.total + tok] =
                sum > 0.f ? (top + log2f(sum)) * 0.69314718055994530942f : -INFINITY;
        }
    }
}

// Rounded up to whole 256-byte steps of the workspace.
template <typename T>
T *take(uintptr_t &at, size_t n) {
    T *p = reinterpret_cast<T *>(at);
    at += (n * sizeof(T) + 255) & ~size_t(255);
    return p;
}

int at_most(long long want, int most) { return (int)(want < 1 ? 1 : want < most ? want : most); }

template <int D, bool BF16>
cudaError_t launch_few_t(const PagedArgs &a, const PagedPlan &w, bool after, cudaStream_t st) {
    using L = FewLayout<D>;
    CUtensorMap tk, tv;
    if (!make_tmap_pages_4d(&tk, a.k_cache, BF16, D, a.page_size, a.num_pages, a.Hkv, L::TK) ||
        !make_tmap_pages_4d(&tv, a.v_cache, BF16, D, a.page_size, a.num_pages, a.Hkv, L::TK))
        return cudaErrorInvalidValue;
    FewParams p;
    p.a = a;
    p.group = fast_div(a.Hq / a.Hkv);
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.status = device_status_ptr();
    p.part = w.mixed ? w.beside : w.own;
    p.whole = w.whole ? 1 : 0;
    p.after = after ? 1 : 0;
    p.mixed = w.mixed ? 1 : 0;
    p.joined = w.joined ? 1 : 0;
    const bool eight = (long long)a.max_new * p.group.d <= 8;
    auto kernel = eight ? paged_few_kernel<D, BF16, 1, false> : paged_few_kernel<D, BF16, 2, false>;
    if (a.parents) kernel = eight ? paged_few_kernel<D, BF16, 1, true> : paged_few_kernel<D, BF16, 2, true>;
    return launch_after(kernel, p.part.ctas, kFewThreads, L::ALLOC, st, tk, tv, p);
}

template <int D, bool BF16>
cudaError_t launch_merge_t(const PagedArgs &a, const PagedPlan &w, cudaStream_t st) {
    MergeParams p;
    p.a = a;
    p.own = w.own;
    p.prefix = w.prefix;
    p.beside = w.beside;
    p.heads = fast_div(a.Hq);
    // few rows can have many parts each, many rows have few
    const long long rows = (long long)a.total * a.Hq;
    p.warps = rows <= 1024 ? 8 : rows <= 4096 ? 2 : 1;
    const int cols = rows <= 16384 ? 8 : 16;  // as measured: at the kernel
    const long long per_block = kMergeWarps / p.warps * (32 / (D / cols));
    auto kernel = paged_merge_kernel<D, BF16, false, 8>;
    if (w.prefix.ctas)
        kernel = cols == 8 ? paged_merge_kernel<D, BF16, true, 8> : paged_merge_kernel<D, BF16, true, 16>;
    else if (cols == 16)
        kernel = paged_merge_kernel<D, BF16, false, 16>;
    return launch_after(kernel, at_most((rows + per_block - 1) / per_block, 3 * kSms), 32 * kMergeWarps, 0, st, p);
}

}  // namespace

PagedPlan plan_paged(int B, int total, int max_new, int Hq, int Hkv, int d, int max_pages, int page_size,
                     int prefix_len, int window, void *workspace) {
    PagedPlan w{};
    const int g = Hq / Hkv;
    const size_t rows = (size_t)total * Hq;
    const long long row_blocks = ((long long)total * g + kWideRows - 1) / kWideRows;
    const long long keys = (long long)max_pages * page_size;
    // Rows of a (request, key/value head) pair: up to 16 fill the tile of the
    // few-row kernel, more go to the 256-row one.
    w.few = (long long)max_new * g <= kMaxRows;
    uintptr_t at = reinterpret_cast<uintptr_t>(workspace);
    const int tile = d == 128 ? 64 : 128;
    const long long pairs = (long long)B * Hkv;
    long long few_tiles = (keys + tile - 1) / tile;
    // Blocks of the 256-row kernel, at most.
    const long long most_blocks = (long long)B * (((long long)max_new * g + kWideRows - 1) / kWideRows);
    const long long blocks = row_blocks + B < most_blocks ? row_blocks + B : most_blocks;
    // Where the requests have a quarter of the longest one's rows or less on
    // average, most are short: the few-row kernel takes those.  512 rows and
    // 63 single tokens behind 8k keys each took the 256-row kernel alone 436
    // us, both 349; 4 chunks of 512, where the launch would find nothing, are
    // left to the one.
    w.mixed = !w.few && g <= kMaxRows && 4ll * total <= (long long)B * max_new;
    // A small batch reads the prefix as often as it has requests, in the pass
    // over their own keys: one launch less, and two when nothing is divided.
    // What it reads more than once is up to 2000 tiles (64 MB, 10 us).
    const long long front_tiles = (prefix_len + tile - 1ll) / tile;
    w.joined = prefix_len > 0 && (w.few || w.mixed ? Hkv * front_tiles * (B - 1) <= 2000 : true);
    const long long wide_front = (prefix_len + kWideKeys - 1ll) / kWideKeys;
    if (w.joined && !w.few) {
        // The 256-row kernel is bound by the tensor cores: the prefix' tiles
        // cost it the same in either pass, but for blocks that the requests'
        // own rows do not fill (up to 128 rows cost 0.55 of 256).  Without the
        // pass, a change of segment (3 tiles) for each of its blocks and four
        // times the rows' fp32 results are saved, at 5 KB in a tile's time.
        // (8 chunks of 512 behind 2k keys: 218 us with the pass, 152 without;
        // 16 of 100 rows behind 8k: 124 and 185.)
        auto part = [](long long n) { return n <= kWideRows / 2 ? 0.55 : 1.0; };
        const double more = (part((long long)max_new * g) * (double)blocks -
                             part((long long)total * g) * (double)row_blocks) * (double)(wide_front * Hkv);
        w.joined = more <= 150.0 + 3.0 * (double)(row_blocks * Hkv) + (double)rows * d / 5000;
    }
    long long wide_tiles = (keys + kWideKeys - 1) / kWideKeys;
    if (w.joined) {
        few_tiles += front_tiles;
        wide_tiles += wide_front;
        prefix_len = 0;
    }
    // a block of up to 256 tokens sees no more than these under a window, in
    // the prefix and behind it
    const long long in_window = window > 0 ? ((long long)window + kWideRows - 1) / kWideKeys + 3 : 1ll << 40;
    w.own_tiles = wide_tiles < in_window ? wide_tiles : in_window;
    w.prefix_tiles = wide_front;
    if (w.few) {
        // A CTA takes whole pairs, with nothing to merge, where the second
        // launch (some 4 us) would cost more than dividing them gains: up to
        // 12 tiles a pair where every pair has a CTA of its own, or up to 8
        // where the CTAs that the last round leaves idle could read little
        // meanwhile.  Measured, us divided and whole, four heads a pair:
        //   8 pairs of 8 tiles 8.8 and 8.5, of 12 8.9 and 10.7, of 16 8.9 and
        //     12.8; 192 (d = 64) of 8 12.6 and 11.7, of 12 15.3 and 15.5, of 16
        //     17.9 and 19.5; 296 of 8 13.5 and 10.6, of 12 22.6 and 20.7
        //   384 of 6 14.3 and 13.4, of 8 17.6 and 18.6; 512 of 8 27.3 and
        //     24.7; 2048 of 4 50.2 and 45.7, of 8 87.7 and 84.9
        const long long seen = window > 0 ? ((long long)window + max_new + tile - 2) / tile + 2 : few_tiles;
        const long long most = seen < few_tiles ? seen : few_tiles;
        const long long idle = (pairs + kMaxCtas - 1) / kMaxCtas * kMaxCtas - pairs;
        w.whole = prefix_len == 0 && (pairs <= kMaxCtas ? most <= 12 : most <= 8 && idle * most <= 800);
        w.own.ctas = at_most(w.whole ? pairs : pairs * few_tiles / kMinUnits, kMaxCtas);
        w.own.slot_rows = kMaxRows;
        if (w.whole) return w;  // no workspace
    } else {
        w.own.ctas = at_most(blocks * Hkv * wide_tiles, kSms);
        w.own.slot_rows = kWideRows;
        if (w.mixed) {
            w.beside.ctas = at_most(pairs * few_tiles / kMinUnits, kMaxCtas);
            w.beside.slot_rows = kMaxRows;
        }
    }
    w.own.code = take<int>(at, rows);
    if (prefix_len > 0) {
        w.prefix.ctas = at_most(row_blocks * Hkv * ((prefix_len + kWideKeys - 1ll) / kWideKeys), kSms);
        w.prefix.slot_rows = kWideRows;
        w.prefix.code = take<int>(at, rows);
        w.own.plane_lse2 = take<float>(at, rows);
        w.own.plane = take<float>(at, rows * d);
        w.prefix.plane_lse2 = take<float>(at, rows);
        w.prefix.plane = take<float>(at, rows * d);
        w.prefix.slot_lse2 = take<float>(at, (size_t)w.prefix.ctas * 2 * kWideRows);
        w.prefix.slot_sum = take<float>(at, (size_t)w.prefix.ctas * 2 * kWideRows);
        w.prefix.slot = take<float>(at, (size_t)w.prefix.ctas * 2 * kWideRows * d);
    }
    w.own.slot_lse2 = take<float>(at, (size_t)w.own.ctas * 2 * w.own.slot_rows);
    if (!w.few) w.own.slot_sum = take<float>(at, (size_t)w.own.ctas * 2 * kWideRows);
    w.own.slot = take<float>(at, (size_t)w.own.ctas * 2 * w.own.slot_rows * d);
    if (w.mixed) {
        w.beside.code = w.own.code;
        w.beside.plane_lse2 = w.own.plane_lse2;
        w.beside.plane = w.own.plane;
        w.beside.slot_lse2 = take<float>(at, (size_t)w.beside.ctas * 2 * kMaxRows);
        w.beside.slot = take<float>(at, (size_t)w.beside.ctas * 2 * kMaxRows * d);
    }
    w.bytes = at - reinterpret_cast<uintptr_t>(workspace);
    return w;
}

cudaError_t launch_paged_few(const PagedArgs &a, const PagedPlan &w, bool after, cudaStream_t st) {
    if (a.d == 128)
        return a.bf16 ? launch_few_t<128, true>(a, w, after, st) : launch_few_t<128, false>(a, w, after, st);
    return a.bf16 ? launch_few_t<64, true>(a, w, after, st) : launch_few_t<64, false>(a, w, after, st);
}

cudaError_t launch_paged_merge(const PagedArgs &a, const PagedPlan &w, cudaStream_t st) {
    if (a.d == 128) return a.bf16 ? launch_merge_t<128, true>(a, w, st) : launch_merge_t<128, false>(a, w, st);
    return a.bf16 ? launch_merge_t<64, true>(a, w, st) : launch_merge_t<64, false>(a, w, st);
}

cudaError_t launch_fwd_paged(const PagedArgs &args, cudaStream_t st) {
    PagedArgs a = args;
    a.shift = 0;
    while ((1 << a.shift) < a.page_size) ++a.shift;
    const PagedPlan w = plan_paged(a.B, a.total, a.max_new, a.Hq, a.Hkv, a.d, a.max_pages, a.page_size, a.prefix_len,
                                   a.window, a.workspace);
    cudaError_t e = cudaSuccess;
    const bool front = w.prefix.ctas > 0;
    if (a.parents && !w.few) {
        a.tree_tiles = tree_tiles(a.max_new);
        a.tree_tokens = tree_tokens(a.Hq / a.Hkv);
        a.tree_words = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(a.workspace) + w.bytes);
        a.tree_depth = reinterpret_cast<int *>(a.tree_words + 2ll * w.own.ctas * a.tree_tokens * a.tree_tiles);
    }
    if (front && (e = launch_paged_wide(a, w, true, false, st)) != cudaSuccess) return e;
    if (!w.few && (e = launch_paged_wide(a, w, false, front, st)) != cudaSuccess) return e;
    if (w.few || w.mixed) e = launch_paged_few(a, w, front || w.mixed, st);
    if (e != cudaSuccess || w.whole) return e;
    return launch_paged_merge(a, w, st);
}

}  // namespace fa
