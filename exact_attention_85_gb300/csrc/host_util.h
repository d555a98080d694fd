// host_util.h -- host-side helpers shared by the launchers: TMA descriptor
// encoding and the launch-argument structs.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace fa {

// Encodes a 3-D tiled TMA descriptor over a dense [dim2][dim1][dim0] tensor
// (dim0 contiguous) with a box of box0 x box1 x 1 elements.  Returns false if
// the driver entry point is unavailable or the encoding is rejected.
bool make_tmap_3d(CUtensorMap *map, const void *base, CUtensorMapDataType dtype, int elem_bytes,
                  uint64_t dim0, uint64_t dim1, uint64_t dim2, uint32_t box0, uint32_t box1,
                  CUtensorMapSwizzle swizzle);

// Row layout of the sequences of one call.
//   dense  (varlen = 0): B sequences of N rows; a tensor with H heads is
//                        [B][H][N][d] and LSE / D are [B][H][N].
//   packed (varlen = 1): B sequences of cu_seqlens[b+1] - cu_seqlens[b] rows
//                        (at most N = max_seqlen) stored back to back,
//                        token-major: [total][H][d]; LSE / D are [H][total].
struct SeqLayout {
    int varlen;
    int B, N;               // sequences, rows per sequence (varlen: the maximum)
    int total;              // varlen: rows of all sequences (cu_seqlens[B])
    const int *cu_seqlens;  // varlen: device [B + 1] prefix sums of the lengths
};

// 3-D tiled TMA descriptor with an explicit three-dimensional box.
bool make_tmap_3d_box(CUtensorMap *map, const void *base, CUtensorMapDataType dtype, int elem_bytes,
                      uint64_t dim0, uint64_t dim1, uint64_t dim2, uint32_t box0, uint32_t box1, uint32_t box2,
                      CUtensorMapSwizzle swizzle);

// TMA descriptor for 64-column x `rows`-row boxes of the 16-bit tensor with
// `heads` heads in layout `lay` (128-byte swizzle).  Dense: coordinates
// (column, row, plane); packed: (column, head, token).
bool make_tmap_tiles(CUtensorMap *map, const void *base, CUtensorMapDataType dtype, int d, const SeqLayout &lay,
                     int heads, uint32_t rows);

// TMA descriptor over the pages of a 16-bit cache [num_pages][heads]
// [page_size][d]: boxes of 64 columns and `keys` rows, or a page's if those
// are fewer; coordinates (column, row of the page, page * heads + head).
bool make_tmap_pages(CUtensorMap *map, const void *base, bool bf16, int d, int page_size, int num_pages, int heads,
                     int keys);

// The same with both 64-column halves of a page's rows in one box, one behind
// the other: coordinates (column, row of the page, half, page * heads + head).
bool make_tmap_pages_4d(CUtensorMap *map, const void *base, bool bf16, int d, int page_size, int num_pages, int heads,
                        int keys);

// TMA descriptor over token-major rows [total][heads][group][d], 16-bit:
// boxes of 64 columns, all of a group and `tokens` tokens; coordinates
// (column, row of the group, group, token).  group * tokens at most 256.
bool make_tmap_rows(CUtensorMap *map, const void *base, bool bf16, int d, int group, int heads, int total, int tokens);

// Dynamic shared memory of a launch.  What a kernel may ask for is an
// attribute of the kernel, seen by every thread: where the bytes depend on
// the call, each call sets it to the `most` that any has, so that a call
// beside it finds its own still allowed.
struct DynSmem {
    size_t bytes, most;
    DynSmem(size_t n) : bytes(n), most(n) {}
    DynSmem(size_t n, size_t most_) : bytes(n), most(most_) {}
};

// Launches `kernel` with `smem` bytes of dynamic shared memory, allowed to
// start before the stream's previous kernel has finished (programmatic
// dependent launch): at its end, or once all its CTAs have said so.  The
// kernel waits for it (griddepcontrol.wait) before it touches memory, so that
// only launch and set-up overlap.
// `cluster`: CTAs of a cluster (1: none).
template <typename... P, typename... A>
cudaError_t launch_cluster_after(void (*kernel)(P...), unsigned grid, unsigned cluster, unsigned threads, DynSmem smem,
                                 cudaStream_t st, const A &...args) {
    // A kernel gets 48 KB without being asked, its static bytes among them:
    // 16 KB are left for those.
    if (smem.bytes > 32 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem.most);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem.bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), unsigned grid, unsigned threads, DynSmem smem, cudaStream_t st,
                         const A &...args) {
    return launch_cluster_after(kernel, grid, 1, threads, smem, st, args...);
}

// Device address of this library's status words (status.cuh) on the current device
// (looked up once per device and context, cached).
unsigned int *device_status_ptr();

// The CUDA context current on the calling thread (driver handle), or null if
// none is current or the driver entry point is unavailable.  Addresses of
// device symbols are cached per (device, context): after a cudaDeviceReset
// the device's next primary context is a new one and the lookup is redone.
void *current_context();

struct FwdArgs {
    const void *q, *k, *v;
    void *o;
    float *lse;
    int B, Hq, Hkv, N, d, causal;
    float scale;
    bool bf16;
    int window;  // 0: none; > 0: causal sliding window of that many keys
    SeqLayout lay;
    bool o_f32;  // O written as fp32 (debug output), else in the input type
};

struct BwdArgs {
    const void *q, *k, *v, *o, *dO;
    const float *lse;
    void *dq, *dk, *dv;
    int B, Hq, Hkv, N, d, causal;
    float scale;
    bool bf16;
    int window;    // 0: none; > 0: causal sliding window of that many keys
    SeqLayout lay;
    float *D;      // [B][Hq][N] (packed: [Hq][total])
    float *dq_acc; // [B][Hq][N][d]; unused (may be null) by the two-pass backward
};

struct Fp8FwdArgs {
    const void *q8, *k8, *v8;
    const float *q_descale, *k_descale, *v_descale;
    void *o;
    float *lse;
    int B, Hq, Hkv, N, d, causal;
    float scale;
};

struct QuantArgs {
    const void *x;
    const float *signs;
    void *x8;
    float *descale;
    long rows;
    int d;
    float *amax;  // workspace cell
};

cudaError_t launch_fwd(const FwdArgs &a, cudaStream_t st);
// The persistent forward (dense layout, no window, 16-bit output only).
cudaError_t launch_fwd_persist(const FwdArgs &a, cudaStream_t st);
cudaError_t launch_bwd(const BwdArgs &a, cudaStream_t st, bool two_pass);
// The persistent main kernel of the backward (dense layout, atomic dQ, dK and
// dV 32-byte aligned): the step between fa_bwd's D preprocessing and its dQ
// conversion.
cudaError_t launch_bwd_persist_main(const BwdArgs &a, cudaStream_t st);
cudaError_t launch_fwd_fp8(const Fp8FwdArgs &a, cudaStream_t st);
cudaError_t launch_hadamard_quant(const QuantArgs &a, cudaStream_t st);
cudaError_t launch_selftest_wait(int timeout_us, cudaStream_t st);
cudaError_t launch_ex2_rate(float *sink, int blocks, int iters, long long *exps, cudaStream_t st);

}  // namespace fa
