// keep_path.cu -- the accepted path's rows move behind the prefix, in all layers.
//
// A CTA takes one sequence and 256 columns of the caches (a column: 16 bytes of a row of
// one head and layer), reads the path and the pages once, and each thread moves its column
// row by row.  A path is increasing, so path[i] >= i: the row that is stored at i has been
// read if it is one of the path's, and a thread that moves a column in order needs no copy
// aside.  The first entries that are in place are not touched.
//
// Bytes: every moved row, read and written once.  64 sequences, 32 layers of 8 heads of 128
// (44 MB): 10.6 us, 4.2 TB/s, replayed from a graph; before the first row moves a CTA has read the path, then the
// page table, and 2048 CTAs are three rounds of the machine.  (Two columns a thread 12.0 us,
// four 13.9; five, six and eight CTAs an SM instead of four 10.9 to 11.7; CTAs that walk over
// several blocks of columns, the path read once, 13.8 to 17.5.)
#include <cstdint>

#include "../../include/fdec.h"
#include "cache_rows.cuh"
#include "fdec_internal.h"

namespace fdec {

namespace {

template <int N>
__global__ void __launch_bounds__(kColumnThreads)
    keep_path_kernel(const __grid_constant__ KeepParams p, const __grid_constant__ CacheList<N> caches, int blocks) {
    __shared__ int2 s_from[kMaxNodes], s_to[kMaxNodes];
    __shared__ int s_begin, s_end;
    const int tid = threadIdx.x, lane = tid & 31;
    const int b = blockIdx.x / blocks, blk = blockIdx.x % blocks;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid < 32) {
        unsigned flags = 0;
        const int64_t prefix = p.prefix_lens[b];
        int n = p.path_lens[b];
        int node[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            node[h] = lane + 32 * h < p.nodes ? p.path[b * p.path_stride + lane + 32 * h] : p.nodes;
        if (n < 0 || n > p.nodes) {
            flags |= FDEC_DEVERR_SEQ_LEN;
            n = min(max(n, 0), p.nodes);
        }
        if (prefix < 0) {  // (the length stays bad, for whoever reads it next)
            flags |= FDEC_DEVERR_SEQ_LEN;
            n = 0;
        }
        // up to the first entry that is out of order; the first that moves
        const int below0 = __shfl_up_sync(0xffffffffu, node[0], 1), last0 = __shfl_sync(0xffffffffu, node[0], 31);
        const int below1 = __shfl_up_sync(0xffffffffu, node[1], 1);
        uint64_t bad = 0, moves = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int below = h == 0 ? (lane == 0 ? -1 : below0) : (lane == 0 ? last0 : below1);
            const bool wrong = node[h] <= below || node[h] >= p.nodes;
            bad |= static_cast<uint64_t>(__ballot_sync(0xffffffffu, wrong)) << (32 * h);
            moves |= static_cast<uint64_t>(__ballot_sync(0xffffffffu, node[h] != lane + 32 * h)) << (32 * h);
        }
        const int good = bad == 0 ? kMaxNodes : __ffsll(static_cast<long long>(bad)) - 1;
        if (good < n) {
            flags |= FDEC_DEVERR_TREE;
            n = good;
        }
        const int begin = moves == 0 ? n : min(n, __ffsll(static_cast<long long>(moves)) - 1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = lane + 32 * h;
            if (i < begin || i >= n) continue;
            int2 at[2];
            bool ok = true;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int64_t pos = prefix + (k == 0 ? node[h] : i), pi = pos >> p.page_shift;
                at[k] = make_int2(-1, static_cast<int>(pos & ((1 << p.page_shift) - 1)));
                if (pi >= p.pt_cols) {
                    flags |= FDEC_DEVERR_SEQ_LEN;
                    ok = false;
                } else {
                    at[k].x = p.page_table[b * p.pt_stride + pi];
                    if (at[k].x < 0 || at[k].x >= p.num_pages) {
                        flags |= FDEC_DEVERR_PAGE_ID;
                        ok = false;
                    }
                }
            }
            if (!ok) at[0].x = -1;
            s_from[i] = at[0];
            s_to[i] = at[1];
        }
        if (lane == 0) {
            s_begin = begin;
            s_end = n;
            if (blk == 0) p.seq_lens[b] = static_cast<int32_t>(min(prefix + n, static_cast<int64_t>(INT32_MAX)));
        }
        if (blk == 0 && flags != 0 && p.err != nullptr) atomicOr(p.err, flags);
    }
    __syncthreads();
    const int begin = s_begin, end = s_end;
    if (begin >= end) return;
    const CacheRows& c = cache_of(caches, blk);
    const auto from = [&](int i) { return s_from[i]; };
    const auto to = [&](int i) { return s_to[i]; };
    if (c.wide)
        move_columns<uint4>(c, blk, begin, end, from, to);
    else
        move_columns<uint2>(c, blk, begin, end, from, to);
}

template <int N>
cudaError_t launch_keep(const KeepParams& p, const CacheList<kMaxCaches>& caches, cudaStream_t s) {
    const int64_t blocks = column_blocks(caches);
    if (blocks * p.batch > INT32_MAX) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks * p.batch), 1, 1);
    cfg.blockDim = dim3(kColumnThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, keep_path_kernel<N>, p, shorter<N>(caches), static_cast<int>(blocks));
}

}  // namespace

cudaError_t launch_keep_path(const KeepParams& p, const CacheList<kMaxCaches>& caches, cudaStream_t s) {
    return caches.n <= 2 ? launch_keep<2>(p, caches, s) : launch_keep<kMaxCaches>(p, caches, s);
}

}  // namespace fdec
