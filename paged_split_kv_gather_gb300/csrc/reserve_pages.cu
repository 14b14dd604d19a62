// reserve_pages.cu -- pages for new lengths, forks of sequences, pages of their own for
// shared ones.
//
// The page tables and lengths say which pages are in use; nothing else is kept, so
// nothing can go out of step with them.  Three launches, one more for large pools, one more where
// there are rows to copy: clear two bit sets of a bit a page; mark every page that an entry in use names (the second set: pages that
// two name); then each sequence finds its pages for itself: how many pages the sequences
// before it need, from the lengths, and which bits are its own, from the pages in use of every
// 1024 and the first bit set.  Those numbers come from a launch of their own for pools above
// 131072 pages (from the marking's atomics they cost 45 us, for 256 sequences and a million
// pages, each CTA reading all bits 9 us); below, every CTA counts for itself.
// The rows that a fork or a shared last page needs are copied last.
// (Each sequence goes through the requests of those before it: of a page each, called one by one, 64 sequences take
// 13.4 us, 256 14.6, 1024 21, 4096 60 and 65536 7.3 ms.)
//
// Bytes: the entries in use, a bit or two a page, and the copied rows, read and written.  64
// sequences and 65536 pages: 8.9 us, the latencies of three dependent launches (clear 1,
// mark 3, assign 3.5); 256 sequences of 2049 entries and a million pages: 14.8, the marks'
// atomics among them; 64 forks in 16 layers: 13.9, of them 7.4 the copies (63 MB, 8.5 TB/s
// of reads and writes that the L2 holds in part).
#include <algorithm>
#include <cstdint>

#include "../../include/fdec.h"
#include "cache_rows.cuh"
#include "fdec_internal.h"

namespace fdec {

namespace {

constexpr int kReserveThreads = kColumnThreads;

// What a sequence asks for.  Entries [first, want) of its row get new pages; a copy fills
// the first of them with `part` rows of page `last`.
struct Request {
    int64_t first, want;
    int source;
    int part;
    bool bad;
    __device__ __forceinline__ int64_t need() const { return want > first ? want - first : 0; }
};

__device__ __forceinline__ bool length_ok(const ReserveParams& p, int64_t n) {
    return n >= 0 && n <= p.pt_cols << p.page_shift;
}

// The sequence's source (itself if none) and the positions it begins with; source -1: bad.
__device__ __forceinline__ int source_of(const ReserveParams& p, int b, int64_t* kept, int64_t* own) {
    const int64_t len = p.seq_lens[b], want = p.new_lens[b];
    int a = p.sources != nullptr ? p.sources[b] : -1;
    if (a < 0) a = b;
    *own = len;
    if (!length_ok(p, len) || !length_ok(p, want) || a >= p.batch) return -1;
    if (a == b) {
        *kept = min(len, want);
        return b;
    }
    const int64_t theirs = p.seq_lens[a];
    const int up = p.sources[a];
    if (len != 0 || !length_ok(p, theirs) || (up >= 0 && up != a)) return -1;
    *kept = min(theirs, want);
    return a;
}

__device__ __forceinline__ Request request_of(const ReserveParams& p, int b) {
    Request r;
    int64_t kept = 0, own = 0;
    r.source = source_of(p, b, &kept, &own);
    r.bad = r.source < 0;
    r.first = r.want = 0;
    r.part = 0;
    if (r.bad) return r;
    const int64_t mask = (1 << p.page_shift) - 1, want = p.new_lens[b];
    r.want = (want + mask) >> p.page_shift;
    if (r.source != b) {
        r.first = kept >> p.page_shift;
        r.part = static_cast<int>(kept & mask);
    } else if (want <= own) {
        r.first = r.want;
    } else {
        r.first = (own + mask) >> p.page_shift;
        const int page = own & mask ? p.last_page[b] : -1;
        if (page >= 0 && (p.shared[page >> 5] >> (page & 31) & 1)) {
            r.first = own >> p.page_shift;
            r.part = static_cast<int>(own & mask);
        }
    }
    return r;
}

__global__ void __launch_bounds__(kReserveThreads) reserve_clear_kernel(const ReserveParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int i = blockIdx.x * kReserveThreads + threadIdx.x; i < p.words; i += gridDim.x * kReserveThreads) {
        p.used[i] = 0;
        p.shared[i] = 0;
    }
}

__global__ void __launch_bounds__(kReserveThreads) reserve_mark_kernel(const ReserveParams p, int blocks) {
    constexpr int U = 4;
    const int b = blockIdx.x / blocks, blk = blockIdx.x % blocks;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int32_t* row = p.page_table + b * p.pt_stride;
    const int64_t room = p.pt_cols << p.page_shift;
    int64_t len = p.seq_lens[b];
    unsigned flags = 0;
    if (!length_ok(p, len)) {
        flags |= FDEC_DEVERR_SEQ_LEN;
        len = len < 0 ? 0 : room;
    }
    const int64_t entries = (len + (1 << p.page_shift) - 1) >> p.page_shift;
    for (int64_t j0 = static_cast<int64_t>(blk) * kReserveThreads * U + threadIdx.x; j0 < entries;
         j0 += static_cast<int64_t>(blocks) * kReserveThreads * U) {
        int page[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t j = j0 + u * kReserveThreads;
            page[u] = j < entries ? row[j] : -2;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (page[u] == -2 && j0 + u * kReserveThreads >= entries) continue;
            if (page[u] < 0 || page[u] >= p.num_pages) {
                flags |= FDEC_DEVERR_PAGE_ID;
                continue;
            }
            const unsigned bit = 1u << (page[u] & 31);
            if (atomicOr(p.used + (page[u] >> 5), bit) & bit) atomicOr(p.shared + (page[u] >> 5), bit);
        }
    }
    if (blk == 0 && threadIdx.x == 0) {
        // the page that a copy would read: the rows of the call are written only after this launch
        int64_t kept = 0, own = 0;
        const int a = source_of(p, b, &kept, &own);
        int page = -1;
        if (a >= 0 && kept & ((1 << p.page_shift) - 1)) page = p.page_table[a * p.pt_stride + (kept >> p.page_shift)];
        p.last_page[b] = page >= 0 && page < p.num_pages ? page : -1;
    }
    if (flags != 0 && p.err != nullptr) atomicOr(p.err, flags);
}

// Up to so many blocks of pages (131072 pages) every CTA counts what is in use for itself.
constexpr int kOwnBlocks = 128;

// Pages in use of block j: a warp, a word of the bit set for each lane.
__device__ __forceinline__ int taken_of(const ReserveParams& p, int j) {
    const int w = j * (kCountedPages / 32) + (threadIdx.x & 31);
    return __reduce_add_sync(0xffffffffu, w < p.words ? __popc(p.used[w]) : 0);
}

__global__ void __launch_bounds__(kReserveThreads) reserve_count_kernel(const ReserveParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warps = gridDim.x * (kReserveThreads / 32);
    for (int j = blockIdx.x * (kReserveThreads / 32) + (threadIdx.x >> 5); j < p.blocks; j += warps) {
        const int taken = taken_of(p, j);
        if ((threadIdx.x & 31) == 0) p.taken[j] = taken;
    }
}

__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* s_part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (lane == 0) s_part[warp] = v;
    __syncthreads();
    int64_t sum = 0;
#pragma unroll
    for (int w = 0; w < kReserveThreads / 32; ++w) sum += s_part[w];
    return sum;
}

__global__ void __launch_bounds__(kReserveThreads) reserve_assign_kernel(const ReserveParams p) {
    __shared__ int64_t s_part[kReserveThreads / 32], s_at;
    __shared__ int s_page, s_block, s_taken[kOwnBlocks];
    __shared__ Request s_request;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // A pool's bits that the CTA counts for itself, all asked for at once.
    const bool own = p.blocks <= kOwnBlocks;
    constexpr int kOwnWords = kOwnBlocks / (kReserveThreads / 32);
    unsigned bits_of[kOwnWords];
#pragma unroll
    for (int k = 0; k < kOwnWords; ++k) {
        const int w = (warp + k * (kReserveThreads / 32)) * (kCountedPages / 32) + lane;
        bits_of[k] = own && w < p.words ? p.used[w] : 0u;
    }
    // what this sequence asks for, and what those before it take
    int64_t start = 0;
    for (int i = tid; i <= b; i += kReserveThreads) {
        const Request q = request_of(p, i);
        if (i == b)
            s_request = q;
        else
            start += q.need();
    }
    start = block_sum(start, s_part);
    const Request r = s_request;
    if (tid == 0 && r.bad && p.err != nullptr) atomicOr(p.err, FDEC_DEVERR_SEQ_LEN);

    bool enough = true;
    if (r.need() > 0) {
        // Free pages by blocks of 1024, a run of blocks for each thread: their number, and the block that holds the
        // sequence's first.
        if (own) {
#pragma unroll
            for (int k = 0; k < kOwnWords; ++k) {
                const int taken = __reduce_add_sync(0xffffffffu, __popc(bits_of[k]));
                if (lane == 0) s_taken[warp + k * (kReserveThreads / 32)] = taken;
            }
            __syncthreads();
        }
        const auto free_of = [&](int j) {
            const int64_t behind = p.num_pages - static_cast<int64_t>(j) * kCountedPages;
            return static_cast<int>(min(behind, static_cast<int64_t>(kCountedPages))) - (own ? s_taken[j] : p.taken[j]);
        };
        const int per = (p.blocks + kReserveThreads - 1) / kReserveThreads;
        const int j0 = min(p.blocks, tid * per), j1 = min(p.blocks, j0 + per);
        int mine = 0;  // (at most 2^26)
        for (int j = j0; j < j1; ++j) mine += free_of(j);
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        __syncthreads();
        if (lane == 31) s_part[warp] = upto;
        __syncthreads();
        int64_t total = 0, at = upto - mine;
#pragma unroll
        for (int w = 0; w < kReserveThreads / 32; ++w) {
            if (w < warp) at += s_part[w];
            total += s_part[w];
        }
        const int64_t end = start + r.need();
        enough = end <= total;
        if (enough && at <= start && start < at + mine) {
            int j = j0;
            for (int here; at + (here = free_of(j)) <= start; ++j) at += here;
            s_block = j;
            s_at = at;
        }
        __syncthreads();
        if (enough) {  // from there on, a block for each warp in turn
            at = s_at;
            for (int j = s_block; at < end; ++j) {
                if ((j - s_block) % (kReserveThreads / 32) == warp) {
                    const int w = j * (kCountedPages / 32) + lane;
                    const int64_t behind = p.num_pages - static_cast<int64_t>(w) * 32;  // bits from this word on
                    unsigned bits = behind <= 0 ? 0u : ~p.used[w] & (behind >= 32 ? 0xffffffffu : (1u << behind) - 1);
                    int before = __popc(bits);
                    const int count = before;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int x = __shfl_up_sync(0xffffffffu, before, o);
                        if (lane >= o) before += x;
                    }
                    int64_t i = at + before - count;
                    for (; bits != 0 && i < end; bits &= bits - 1, ++i) {
                        if (i < start) continue;
                        const int page = w * 32 + __ffs(bits) - 1;
                        p.page_table[b * p.pt_stride + r.first + (i - start)] = page;
                        if (i == start) s_page = page;
                    }
                }
                at += free_of(j);
            }
        }
    }
    if (tid == 0) {
        p.granted[b] = r.bad || !enough ? p.seq_lens[b] : p.new_lens[b];
        if (!enough && p.err != nullptr) atomicOr(p.err, FDEC_DEVERR_NO_PAGES);
    }
    if (!r.bad && enough && r.source != b)  // a fork shares the full pages
        for (int64_t j = tid; j < r.first; j += kReserveThreads)
            p.page_table[b * p.pt_stride + j] = p.page_table[r.source * p.pt_stride + j];
    __syncthreads();
    if (tid == 0) {
        const int of = p.last_page[b];  // (a bad one has been flagged)
        const bool copies = !r.bad && enough && r.part > 0 && r.need() > 0 && of >= 0;
        p.copies[b] = copies ? make_int4(of, s_page, r.part, 0) : make_int4(0, 0, 0, 0);
    }
}

template <int N>
__global__ void __launch_bounds__(kColumnThreads)
    reserve_copy_kernel(const __grid_constant__ ReserveParams p, const __grid_constant__ CacheList<N> caches, int blocks) {
    const int b = blockIdx.x / blocks, blk = blockIdx.x % blocks;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 copy = p.copies[b];
    if (copy.z == 0) return;
    const CacheRows& c = cache_of(caches, blk);
    const auto from = [&](int i) { return make_int2(copy.x, i); };
    const auto to = [&](int i) { return make_int2(copy.y, i); };
    if (c.wide)
        move_columns<uint4>(c, blk, 0, copy.z, from, to);
    else
        move_columns<uint2>(c, blk, 0, copy.z, from, to);
}

template <typename Kernel, typename... Args>
cudaError_t launch(Kernel kernel, int64_t grid, cudaStream_t s, const Args&... args) {
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(kReserveThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int N>
cudaError_t launch_copy(const ReserveParams& p, const CacheList<kMaxCaches>& caches, cudaStream_t s) {
    const int64_t blocks = column_blocks(caches);
    return launch(reserve_copy_kernel<N>, blocks * p.batch, s, p, shorter<N>(caches), static_cast<int>(blocks));
}

}  // namespace

cudaError_t launch_reserve_pages(const ReserveParams& p, const CacheList<kMaxCaches>& caches, int num_sms,
                                 cudaStream_t s) {
    const int64_t clear = std::min<int64_t>((p.words + kReserveThreads - 1) / kReserveThreads, num_sms * 4);
    cudaError_t e = launch(reserve_clear_kernel, clear, s, p);
    if (e != cudaSuccess) return e;
    const int64_t row_blocks = (p.pt_cols + kReserveThreads * 4 - 1) / (kReserveThreads * 4);
    const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>(row_blocks, num_sms * 16 / p.batch));
    e = launch(reserve_mark_kernel, blocks * p.batch, s, p, static_cast<int>(blocks));
    if (e != cudaSuccess) return e;
    if (p.blocks > kOwnBlocks) {
        e = launch(reserve_count_kernel, std::min<int64_t>((p.blocks + 7) / 8, num_sms * 4), s, p);
        if (e != cudaSuccess) return e;
    }
    e = launch(reserve_assign_kernel, p.batch, s, p);
    if (e != cudaSuccess || caches.n == 0) return e;
    return caches.n <= 2 ? launch_copy<2>(p, caches, s) : launch_copy<kMaxCaches>(p, caches, s);
}

}  // namespace fdec
