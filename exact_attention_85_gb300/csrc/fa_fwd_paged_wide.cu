// fa_fwd_paged_wide.cu -- forward attention from a paged key/value cache for
// many query rows: prompts read in by chunks, and the rows of a whole batch
// against a prefix that all its requests share.
//
// One CTA owns 256 query rows of one key/value head and a range of its key
// tiles.  A row is a (token, query head) pair: the g = Hq / Hkv heads that
// read the key/value head are neighbouring rows of the tile, so grouped
// heads share every K/V tile that is read, and with a shared prefix so do all
// requests (their rows stand one behind the other in q).  The loop is that of
// the dense forward (fa_fwd.cu): two 128-row Q tiles A and B walk the same
// K/V stream, their softmax warpgroups take turns on the tensor cores, O is
// rescaled lazily and exactly, and P is read from tensor memory.  What
// differs: K/V tiles are gathered page by page (one TMA box per page and
// 64-column half), Q rows are copied into the swizzled operand layout by the
// softmax threads, every row has its own visible range of keys, and a CTA may
// take only part of the key tiles and leave (O~ / l, log2 sum) for a merge.
//   warps 0-3 softmax + epilogue of tile A, 4-7 of tile B, 8 producer,
//   9 MMA issuer (owns the tensor memory)
#include "../../include/fa.h"
#include "host_util.h"
#include "paged.h"
#include "paged_dev.cuh"
#include "ptx.cuh"

namespace fa {

namespace {

constexpr int kBM = 128, kBN = 128;
constexpr int kRows = 2 * kBM;
constexpr int kThreads = 320;
constexpr int kProducerWarp = 8, kMmaWarp = 9;
constexpr float kRescaleThreshold = 8.0f;
constexpr uint32_t kColS = 0, kColO = 256;  // + 128 per tile

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
    // p_full[2], o_final[2], drain
    static constexpr int NBAR = 1 + 2 * KS + 2 * VS + 2 + 2 + 2 + 1;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int BYTES = OFF_MISC + 48;
    static constexpr int ALLOC = BYTES + 1024;
    static_assert(ALLOC <= 227 * 1024, "shared memory");
};

struct WideParams {
    PagedArgs a;
    int shift;        // log2(page_size)
    int group;        // query heads per key/value head
    int prefix;       // 1: rows of the whole batch against the shared prefix
    int blocks;       // row blocks (upper bound)
    int splits;       // key ranges
    float *part_o;    // [splits][total][Hq][D], or null: O and LSE are final
    float *part_lse2; // [splits][total][Hq]
    float scale_log2;
    unsigned int *status;
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

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    paged_wide_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const WideParams p) {
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
    uint64_t *drain = o_final + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::OFF_MISC + 4);
    int *block_at = reinterpret_cast<int *>(smem + L::OFF_MISC + 8);  // request, block within it
    int *low_key = reinterpret_cast<int *>(smem + L::OFF_MISC + 16);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // (key range, key/value head, row block): the key ranges of one block are
    // far apart in the grid, neighbouring CTAs read the same keys
    const int hk = (blockIdx.x / p.blocks) % p.a.Hkv;
    const int split = blockIdx.x / p.blocks / p.a.Hkv;
    const int block = blockIdx.x % p.blocks;

    // ------------------------------------------- the block's rows and keys
    int row0 = 0, n = 0, len = 0, r0 = 0;  // request's rows and keys; first row of the block
    const int *table = p.a.prefix_pages;
    if (p.prefix) {
        n = p.a.cu_seqlens ? p.a.cu_seqlens[p.a.B] : p.a.B;
        // offsets that end outside q are reported with their request; the
        // sound ones may have rows anywhere
        if (n < 0 || n > p.a.total) n = p.a.total;
        len = p.a.prefix_len;
        r0 = block * kRows;
    } else {
        // blocks are numbered through the requests' rows
        if (warp == 0) {
            if (lane == 0) block_at[0] = -1;
            int at = 0;  // blocks before request b
            for (int b = 0; b < p.a.B; b += 32) {
                Request r;
                int mine = 0;
                if (b + lane < p.a.B) {
                    if (!load_request(p.a, p.shift, b + lane, r)) {
                        if (blockIdx.x == 0) record_bad_args(p.status);
                    } else {
                        mine = (int)(((long long)r.n * p.group + kRows - 1) / kRows);
                    }
                }
                int incl = mine;
#pragma unroll
                for (int s = 1; s < 32; s <<= 1) {
                    const int x = __shfl_up_sync(0xffffffffu, incl, s);
                    if (lane >= s) incl += x;
                }
                const unsigned past = __ballot_sync(0xffffffffu, at + incl > block);
                if (past) {
                    if (lane == __ffs(past) - 1) {
                        block_at[0] = b + lane;
                        block_at[1] = block - (at + incl - mine);
                    }
                    if (blockIdx.x != 0) break;  // CTA 0 goes through all, to report bad ones
                    at = -0x40000000;
                    continue;
                }
                at += __shfl_sync(0xffffffffu, incl, 31);
            }
        }
        __syncthreads();
        const int b = block_at[0];
        if (b < 0) return;  // more blocks than the batch has: nothing started yet
        Request r;
        load_request(p.a, p.shift, b, r);
        row0 = r.row0;
        n = r.n;
        len = r.len;
        r0 = block_at[1] * kRows;
        table = p.a.block_table + (size_t)b * p.a.max_pages;
    }
    const int rows = (int)min((long long)n * p.group - r0, (long long)kRows);  // of this block
    if (rows <= 0) return;
    const int t_first = r0 / p.group, t_last = (r0 + rows - 1) / p.group;

    // this thread's row (softmax warps): where it is and which keys it sees
    const int row = threadIdx.x;
    const bool valid = row < rows;
    int tok = 0, head = 0, hi = 0x7FFFFFFF, lo = -0x7FFFFFFF;
    if (valid) {
        const int t = (r0 + row) / p.group;
        head = hk * p.group + (r0 + row) - t * p.group;
        tok = row0 + t;
        if (p.prefix) {
            const int b = request_of(p.a, tok);
            Request r;
            if (load_request(p.a, p.shift, b, r)) {
                hi = p.a.prefix_len + r.len - r.n + (tok - r.row0) + 1;
                lo = p.a.window > 0 ? hi - p.a.window : 0;
            }
        } else {
            hi = len - n + t + 1;
            lo = p.a.window > 0 ? hi - p.a.window : 0;
        }
    }
    // keys some row of the block sees
    int key_lo = 0, key_hi = len;
    if (p.prefix) {
        if (p.a.window > 0) {
            if (threadIdx.x == 0) *low_key = 0x7FFFFFFF;
            __syncthreads();
            if (valid) atomicMin(low_key, max(0, min(lo, len)));
            __syncthreads();
            key_lo = *low_key;
        }
    } else {
        key_hi = max(0, len - n + t_last + 1);
        if (p.a.window > 0) key_lo = max(0, len - n + t_first + 1 - p.a.window);
    }
    const int t0 = key_lo / kBN;
    const int tiles = max(0, (key_hi + kBN - 1) / kBN - t0);
    // this CTA's tiles; with nothing to see, one fully masked tile keeps the
    // path the same
    const int j0 = t0 + (int)((long long)tiles * split / p.splits);
    const int j1 = t0 + (int)((long long)tiles * (split + 1) / p.splits);
    const int nj = j1 - j0;
    const bool two = rows > kBM;

    if (nj == 0) {  // uniform: an empty range (few tiles, many ranges)
        if (valid) {
            if (p.part_o) {
                p.part_lse2[((size_t)split * p.a.total + tok) * p.a.Hq + head] = -INFINITY;
            } else {
                uint4 *o = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.a.o) + ((size_t)tok * p.a.Hq + head) * D);
                for (int c = 0; c < D / 8; ++c) o[c] = make_uint4(0, 0, 0, 0);
                p.a.lse[(size_t)head * p.a.total + tok] = -INFINITY;
            }
        }
        return;
    }

    if (threadIdx.x == 0) {
        mbar_init(q_full, 2 * kBM);
        for (int s = 0; s < L::KS; ++s) { mbar_init(&k_full[s], 1); mbar_init(&k_empty[s], 1); }
        for (int s = 0; s < L::VS; ++s) { mbar_init(&v_full[s], 1); mbar_init(&v_empty[s], 1); }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&s_full[x], 1);
            mbar_init(&p_full[x], kBM);
            mbar_init(&o_final[x], 1);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == kProducerWarp) {
        // ------------------------------------------------------ TMA producer
        if (lane == 0) {
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_v);
        }
        const int page_keys = min(1 << p.shift, kBN);
        const int box_bytes = page_keys * 128;
        const int half = lane % L::NBOX, sub = lane / L::NBOX;
        const bool boxed = lane < L::NBOX * (kBN / page_keys);
        int done = 0;
        bool v_missing = false;
        for (int u = 0; u < nj; ++u) {
            // pages that hold no key of the block's range are not looked up
            const int key0 = (j0 + u) * kBN + sub * page_keys;
            const bool live = boxed && key0 < key_hi && key0 + page_keys > key_lo;
            int page = 0;
            if (live) {
                page = table[key0 >> p.shift];
                if (page < 0 || page >= p.a.num_pages) {
                    record_bad_args(p.status);
                    page = p.a.num_pages;  // out of the tensor: the copy fills zeros
                }
            }
            const int bytes = __popc(__ballot_sync(0xffffffffu, live)) * box_bytes;
            const int ks = u % L::KS, vs = u % L::VS;
            bool ok = u < L::KS || mbar_wait(&k_empty[ks], ((u / L::KS) + 1) & 1, abort_flag, p.status, 31);
            if (!__all_sync(0xffffffffu, ok)) break;
            if (lane == 0) mbar_arrive_expect_tx(&k_full[ks], bytes);
            __syncwarp();
            const int in_page = key0 & ((1 << p.shift) - 1);
            if (live)
                tma_load_3d(smem + L::OFF_K + ks * L::TILE + half * L::BOX + sub * box_bytes, &tm_k, &k_full[ks],
                            half * 64, in_page, page * p.a.Hkv + hk);
            ok = u < L::VS || mbar_wait(&v_empty[vs], ((u / L::VS) + 1) & 1, abort_flag, p.status, 32);
            if (!__all_sync(0xffffffffu, ok)) {
                v_missing = true;
                break;
            }
            if (lane == 0) mbar_arrive_expect_tx(&v_full[vs], bytes);
            __syncwarp();
            if (live)
                tma_load_3d(smem + L::OFF_V + vs * L::TILE + half * L::BOX + sub * box_bytes, &tm_v, &v_full[vs],
                            half * 64, in_page, page * p.a.Hkv + hk);
            ++done;
        }
        if (done < nj && lane == 0) {
            // given up: let copies in flight land before the CTA exits
            const int nk = done + (v_missing ? 1 : 0);
            for (int u = max(0, nk - L::KS); u < nk; ++u)
                mbar_wait_drain(&k_full[u % L::KS], (u / L::KS) & 1, 10000000ull);
            for (int u = max(0, done - L::VS); u < done; ++u)
                mbar_wait_drain(&v_full[u % L::VS], (u / L::VS) & 1, 10000000ull);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // -------------------------------------------------------- MMA issuer
        // lane 0 issues; the whole warp follows, to clear V rows (below)
        constexpr uint32_t fmt = BF16 ? 1u : 0u;
        constexpr uint32_t idesc_s = make_idesc(kBM, kBN, fmt, false, false);
        constexpr uint32_t idesc_pv = make_idesc(kBM, D, fmt, false, true);
        const uint64_t q_desc0 = make_sdesc_sw128(smem_u32(smem + L::OFF_Q), 16, 1024);
        const uint64_t k_desc0 = make_sdesc_sw128(smem_u32(smem + L::OFF_K), 16, 1024);
        const uint64_t v_desc0 = make_sdesc_sw128(smem_u32(smem + L::OFF_V), L::BOX, 1024);
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
        auto issue_pv = [&](int x, int u) {
            const uint64_t v_desc = sdesc_advance(v_desc0, (u % L::VS) * L::TILE);
            const uint32_t p_col = tmem + kColS + x * 128;
#pragma unroll
            for (int kk = 0; kk < kBN / 16; ++kk)
                mma_f16_ts(tmem + kColO + x * 128, p_col + kk * 8, sdesc_advance(v_desc, kk * 2048), idesc_pv,
                           (u > 0 || kk > 0) ? 1u : 0u);
        };
        auto wait = [&](uint64_t *bar, int parity, int site) -> bool {
            const bool got = mbar_wait(bar, parity, abort_flag, p.status, site);
            tc_fence_after();
            return __all_sync(0xffffffffu, got);
        };
        bool ok = wait(q_full, 0, 33) && wait(&k_full[0], 0, 34);
        if (ok && lane == 0) {
            issue_s(0, 0);
            if (two) issue_s(1, 0);
            mma_commit(&k_empty[0]);
        }
        for (int u = 0; ok && u < nj; ++u) {
            const int vs = u % L::VS;
            if (!(ok = wait(&v_full[vs], (u / L::VS) & 1, 35))) break;
            const int kv0 = (j0 + u) * kBN;
            if (kv0 < key_lo || kv0 + kBN > key_hi) {
                // V rows that no row of the block sees may hold anything (the
                // rest of a page, a buffer that was not filled), and 0 * NaN
                // is NaN: clear them
                uint8_t *v = smem + L::OFF_V + vs * L::TILE;
                for (int i = lane; i < kBN * 8 * L::NBOX; i += 32) {
                    const int key = kv0 + ((i >> 3) & (kBN - 1));
                    if (key < key_lo || key >= key_hi) reinterpret_cast<uint4 *>(v)[i] = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
            if (!(ok = wait(&p_full[0], u & 1, 36))) break;
            if (lane == 0) {
                issue_pv(0, u);
                if (u + 1 == nj) mma_commit(&o_final[0]);
            }
            if (u + 1 < nj) {
                if (!(ok = wait(&k_full[(u + 1) % L::KS], ((u + 1) / L::KS) & 1, 34))) break;
                if (lane == 0) {
                    issue_s(0, u + 1);
                    if (!two) mma_commit(&k_empty[(u + 1) % L::KS]);
                }
            }
            if (two) {
                if (!(ok = wait(&p_full[1], u & 1, 36))) break;
                if (lane == 0) {
                    issue_pv(1, u);
                    if (u + 1 == nj) mma_commit(&o_final[1]);
                }
            }
            if (lane == 0) {
                mma_commit(&v_empty[vs]);
                if (two && u + 1 < nj) {
                    issue_s(1, u + 1);
                    mma_commit(&k_empty[(u + 1) % L::KS]);
                }
            }
            __syncwarp();
        }
        if (lane == 0) {
            // every MMA issued above has completed once `drain` flips
            mma_commit(drain);
            mbar_wait_drain(drain, 0, 100000000ull);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ softmax + epilogue
        const int x = warp >> 2;
        const int quarter = warp & 3;
        const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t col_s = kColS + x * 128, col_o = kColO + x * 128;
        {
            // Q into the operand layout: 16-byte pieces, a row's pieces by
            // neighbouring lanes; rows past the block's own are zeros
            constexpr int CH = D / 8;
            for (int i = threadIdx.x; i < kRows * CH; i += kRows) {
                const int r = i / CH, ch = i % CH;
                uint4 w = make_uint4(0, 0, 0, 0);
                if (r < rows) {
                    const int t = (r0 + r) / p.group;
                    w = static_cast<const uint4 *>(
                        p.a.q)[((size_t)(row0 + t) * p.a.Hq + hk * p.group + (r0 + r) - t * p.group) * CH + ch];
                }
                *reinterpret_cast<uint4 *>(smem + L::OFF_Q + (r >> 7) * L::TILE + (ch >> 3) * L::BOX +
                                           (r & 127) * 128 + (((ch & 7) ^ (r & 7)) << 4)) = w;
            }
            fence_proxy_async_smem();
            mbar_arrive(q_full);
        }
        const float sl2 = p.scale_log2;
        float m_ref = -INFINITY;
        float l_sum = 0.0f;    // sum of the rounded P fed to the MMA: normalises O
        float l_exact = 0.0f;  // sum of the unrounded P: gives L
        const int hi_w = __reduce_min_sync(0xffffffffu, hi), lo_w = __reduce_max_sync(0xffffffffu, lo);
        const bool active = x == 0 || two;
        bool ok = true;
        for (int u = 0; ok && active && u < nj; ++u) {
            const bool got_s = mbar_wait(&s_full[x], u & 1, abort_flag, p.status, 37);
            if (!__all_sync(0xffffffffu, got_s)) { ok = false; break; }
            tc_fence_after();
            uint32_t s[128];
            const uint32_t s_addr = lane_base + col_s;
            tmem_ld_x32(s_addr + 0, s + 0);
            tmem_ld_x32(s_addr + 32, s + 32);
            tmem_ld_x32(s_addr + 64, s + 64);
            tmem_ld_x32(s_addr + 96, s + 96);
            tmem_ld_wait_x32(s + 0);
            tmem_ld_wait_x32(s + 32);
            tmem_ld_wait_x32(s + 64);
            tmem_ld_wait_x32(s + 96);
            const int kv0 = (j0 + u) * kBN;
            if (kv0 + kBN > min(hi_w, key_hi) || kv0 < max(lo_w, key_lo)) {  // uniform in the warp
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
            const float2 neg_m = make_float2(-m_use, -m_use);
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
                        pk[k] = pack_f16x2(p0, p1);
                        pk[k + 1] = pack_f16x2(p2, p3);
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
            if (ok) ok = mbar_wait(&o_final[x], 0, abort_flag, p.status, 38);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
                tc_fence_after();
                const float inv_l = l_sum > 0.f ? 1.0f / l_sum : 0.f;
                const size_t at = (size_t)tok * p.a.Hq + head;
                const size_t part = (size_t)split * p.a.total * p.a.Hq + at;
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t o[32];
                    tmem_ld_x32(lane_base + col_o + c0, o);
                    tmem_ld_wait_x32(o);
#pragma unroll
                    for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * inv_l);
                    if (valid && p.part_o) {
                        uint4 *dst = reinterpret_cast<uint4 *>(p.part_o + part * D + c0);
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            dst[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                    } else if (valid) {
                        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.a.o) + at * D + c0);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t w[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float a = __uint_as_float(o[8 * q + 2 * k]);
                                const float b = __uint_as_float(o[8 * q + 2 * k + 1]);
                                w[k] = BF16 ? pack_bf16x2(a, b) : pack_f16x2(a, b);
                            }
                            dst[q] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    __syncwarp();  // the loads above are the whole warp's
                }
                if (valid) {
                    const float lse2 = l_exact > 0.f ? m_ref + log2f(l_exact) : -INFINITY;
                    if (p.part_o)
                        p.part_lse2[part] = lse2;
                    else
                        p.a.lse[(size_t)head * p.a.total + tok] = lse2 * 0.69314718055994530942f;
                }
            }
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Merges the key ranges of every row: a warp per row and head.
template <int D, bool BF16>
__global__ void __launch_bounds__(128) paged_merge_rows_kernel(const WideParams p) {
    const long long id = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (id >= (long long)p.a.total * p.a.Hq) return;
    const int lane = threadIdx.x & 31;
    const int tok = (int)(id / p.a.Hq), h = (int)(id - (long long)tok * p.a.Hq);
    Request r;
    if (p.a.cu_seqlens ? false : tok >= p.a.B) return;
    if (!load_request(p.a, p.shift, request_of(p.a, tok), r)) return;
    if (tok < r.row0 || tok >= r.row0 + r.n) return;  // a row of no request
    constexpr int E = D / 32;
    float acc[E], top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int s = 0; s < p.splits; ++s) {
        const size_t at = (size_t)s * p.a.total * p.a.Hq + id;
        const float lse2 = p.part_lse2[at];
        if (lse2 == -INFINITY) continue;
        const float to = fmaxf(top, lse2);
        const float a = ex2_approx(top - to), w = ex2_approx(lse2 - to);
        sum = sum * a + w;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * a + w * p.part_o[at * D + lane * E + e];
        top = to;
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    uint16_t *out = static_cast<uint16_t *>(p.a.o) + (size_t)id * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t *>(out + e) =
            BF16 ? pack_bf16x2(acc[e] * inv, acc[e + 1] * inv) : pack_f16x2(acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0)
        p.a.lse[(size_t)h * p.a.total + tok] = sum > 0.f ? (top + log2f(sum)) * 0.69314718055994530942f : -INFINITY;
}

}  // namespace

template <int D, bool BF16>
static cudaError_t launch_wide_t(const PagedArgs &a, int shift, const WidePlan &w, cudaStream_t st) {
    using L = WideLayout<D>;
    const CUtensorMapDataType dt = BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    CUtensorMap tk, tv;
    const uint32_t rows = a.page_size < kBN ? a.page_size : kBN;
    const uint64_t planes = (uint64_t)a.num_pages * a.Hkv;
    if (!make_tmap_3d(&tk, a.k_cache, dt, 2, D, a.page_size, planes, 64, rows, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_tmap_3d(&tv, a.v_cache, dt, 2, D, a.page_size, planes, 64, rows, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    auto kernel = paged_wide_kernel<D, BF16>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::ALLOC);
    if (e != cudaSuccess) return e;
    WideParams p;
    p.a = a;
    p.shift = shift;
    p.group = a.Hq / a.Hkv;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.status = device_status_ptr();
    const size_t plane = (size_t)a.total * a.Hq;
    if (w.prefix_splits) {
        p.prefix = 1;
        p.blocks = w.prefix_blocks;
        p.splits = w.prefix_splits;
        p.part_o = w.part_o;
        p.part_lse2 = w.part_lse2;
        kernel<<<(unsigned)(p.blocks * a.Hkv * p.splits), kThreads, L::ALLOC, st>>>(tk, tv, p);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (!w.own_splits) return cudaSuccess;
    p.prefix = 0;
    p.blocks = w.own_blocks;
    p.splits = w.own_splits;
    const bool direct = w.prefix_splits == 0 && w.own_splits == 1;
    p.part_o = direct ? nullptr : w.part_o + plane * D * w.prefix_splits;
    p.part_lse2 = direct ? nullptr : w.part_lse2 + plane * w.prefix_splits;
    kernel<<<(unsigned)(p.blocks * a.Hkv * p.splits), kThreads, L::ALLOC, st>>>(tk, tv, p);
    if ((e = cudaGetLastError()) != cudaSuccess || direct) return e;
    p.part_o = w.part_o;
    p.part_lse2 = w.part_lse2;
    p.splits = w.prefix_splits + w.own_splits;
    paged_merge_rows_kernel<D, BF16><<<(unsigned)((plane + 3) / 4), 128, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_paged_wide(const PagedArgs &a, int shift, const WidePlan &w, cudaStream_t st) {
    if (a.d == 128) return a.bf16 ? launch_wide_t<128, true>(a, shift, w, st) : launch_wide_t<128, false>(a, shift, w, st);
    return a.bf16 ? launch_wide_t<64, true>(a, shift, w, st) : launch_wide_t<64, false>(a, shift, w, st);
}

}  // namespace fa
