// fa_fwd_paged.cu -- forward attention from a paged key/value cache.
//
// Row i of request b (n_b new rows, len_b keys of its own, of which the last
// n_b belong to the rows) stands at place p = len_b - n_b + i and sees its
// own keys max(0, p - W + 1) .. p; with a shared prefix of P keys in front,
// places count from the prefix' start.  One warp per (row, query head), keys
// one by one with the running maximum and sum of the softmax.
#include "../../include/fa.h"
#include "host_util.h"
#include "paged.h"
#include "ptx.cuh"

namespace fa {

namespace {

struct RowsParams {
    PagedArgs a;
    int shift;  // log2(page_size)
    float scale_log2;
    unsigned int *status;
};

template <int D, bool BF16>
__global__ void __launch_bounds__(128) paged_rows_kernel(const RowsParams p) {
    constexpr int E = D / 32;  // elements a lane holds
    const int lane = threadIdx.x & 31;
    const long long id = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (id >= (long long)p.a.total * p.a.Hq) return;
    const int row = (int)(id / p.a.Hq), h = (int)(id - (long long)row * p.a.Hq);
    const int hk = h / (p.a.Hq / p.a.Hkv);
    // the row's request
    int b, i = 0, n = 1;
    if (!p.a.cu_seqlens) {
        if (row >= p.a.B) return;
        b = row;
    } else {
        const int *cu = p.a.cu_seqlens;
        int lo = 0, hi = p.a.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (cu[mid] <= row) lo = mid; else hi = mid - 1;
        }
        b = lo;
        i = row - cu[b];
        n = cu[b + 1] - cu[b];
        if (i < 0 || i >= n) return;  // behind the last sequence
        if (n > p.a.max_new || cu[b] < 0 || cu[b + 1] > p.a.total) {
            record_bad_args(p.status);
            return;
        }
    }
    const int len = p.a.seq_lens[b];
    if (len < 0 || len > (p.a.max_pages << p.shift)) {
        record_bad_args(p.status);
        return;
    }
    const int P = p.a.prefix_len;
    const int hi = P + len - n + i + 1;  // keys 0 .. hi - 1 from the prefix' start
    const int lo = p.a.window > 0 ? max(0, hi - p.a.window) : 0;
    using T = uint16_t;
    auto widen = [](const T *s, float *x) {
        if constexpr (E == 4) {
            const uint2 w = *reinterpret_cast<const uint2 *>(s);
            const float2 a = unpack2<BF16>(w.x), c = unpack2<BF16>(w.y);
            x[0] = a.x; x[1] = a.y; x[2] = c.x; x[3] = c.y;
        } else {
            const float2 a = unpack2<BF16>(*reinterpret_cast<const uint32_t *>(s));
            x[0] = a.x; x[1] = a.y;
        }
    };
    float q[E], acc[E];
    widen(static_cast<const T *>(p.a.q) + ((size_t)row * p.a.Hq + h) * D + lane * E, q);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    float m = -INFINITY, l = 0.f;
    // with a prefix, a row at a negative place still sees the prefix
    for (int key = lo; key < hi; ++key) {
        const bool front = key < P;
        const int at = front ? key : key - P;
        const int page = front ? p.a.prefix_pages[at >> p.shift]
                               : p.a.block_table[(size_t)b * p.a.max_pages + (at >> p.shift)];
        if (page < 0 || page >= p.a.num_pages) {
            if (lane == 0) record_bad_args(p.status);
            continue;
        }
        const size_t off =
            ((((size_t)page * p.a.Hkv + hk) << p.shift) + (at & ((1 << p.shift) - 1))) * D + lane * E;
        float x[E];
        widen(static_cast<const T *>(p.a.k_cache) + off, x);
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(q[e], x[e], s);
#pragma unroll
        for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
        s *= p.scale_log2;
        if (s > m) {
            const float f = exp2f(m - s);
            l *= f;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] *= f;
            m = s;
        }
        const float w = exp2f(s - m);
        l += w;
        widen(static_cast<const T *>(p.a.v_cache) + off, x);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(w, x[e], acc[e]);
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    T *o = static_cast<T *>(p.a.o) + ((size_t)row * p.a.Hq + h) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t *>(o + e) =
            BF16 ? pack_bf16x2(acc[e] * inv, acc[e + 1] * inv) : pack_f16x2(acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0)
        p.a.lse[(size_t)h * p.a.total + row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994530942f : -INFINITY;
}

}  // namespace

size_t fwd_paged_workspace(int, int, int, int, int, int, int, int, int) { return 256; }

cudaError_t launch_fwd_paged(const PagedArgs &a, cudaStream_t st) {
    RowsParams p{a, 0, a.scale * 1.4426950408889634f, device_status_ptr()};
    while ((1 << p.shift) < a.page_size) ++p.shift;
    const unsigned grid = (unsigned)(((long long)a.total * a.Hq + 3) / 4);
    if (a.d == 128) {
        if (a.bf16) paged_rows_kernel<128, true><<<grid, 128, 0, st>>>(p);
        else paged_rows_kernel<128, false><<<grid, 128, 0, st>>>(p);
    } else {
        if (a.bf16) paged_rows_kernel<64, true><<<grid, 128, 0, st>>>(p);
        else paged_rows_kernel<64, false><<<grid, 128, 0, st>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace fa
